// Entry points of the single operations on rotary positions and the paged 4-bit KV cache
// (include/dllm.h): argument checks, launch shapes and launches. A translation unit of its
// own, so that the engine's kernels and these compile side by side.

#include "dllm.h"

#include <algorithm>
#include <cmath>

#include "attention_kv4.cuh"
#include "attention_kv4_tc.cuh"
#include "kv4.cuh"
#include "rope.cuh"

using namespace dllm;

namespace dllm {
// dllm_set_wait_limit's part in this translation unit (the limit is a constant of each).
cudaError_t kv4_set_wait_limit(unsigned long long ns) { return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns)); }
}  // namespace dllm

namespace {

constexpr int kSMs = 148;
static_assert(kSMs <= kKv4MaxBlocks, "attn_kv4_parts_kernel");

int ceil_div(long a, long b) { return (int)((a + b - 1) / b); }

// Launch with programmatic stream serialisation: the kernel's blocks may be scheduled while
// the kernel before it drains; each waits for that kernel's memory before its first access.
template <typename... KArgs, typename... Args>
cudaError_t launch(cudaStream_t st, void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

int status(cudaError_t e) {
  if (e == cudaSuccess) return DLLM_OK;
  cudaGetLastError();   // a refused launch leaves nothing behind for the next call to report
  return DLLM_E_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
size_t size_of(int type) { return type == DLLM_F32 ? 4 : 2; }

// 16-byte vectors along a head: base and both strides on 16 bytes.
bool vectors(const void* p, int type, long long tok, long long head) {
  const long long per = 16 / (long long)size_of(type);
  return aligned16(p) && tok % per == 0 && head % per == 0;
}

// Whether the rows of an output [T][H][d] are apart: no element lies in two of them, i.e. no two rows i tokens
// and j heads from one another start less than d elements apart. With the strides' signs dropped, j heads on are
// the same as j back for some i.
bool rows_apart(int T, int H, int d, long long tok, long long head) {
  typedef __int128 wide;
  const wide a = tok < 0 ? -(wide)tok : tok, b = head < 0 ? -(wide)head : head;
  if ((T > 1 && a < d) || (H > 1 && b < d)) return false;
  if (T <= 1 || H <= 1 || a >= b * (H - 1) + d || b >= a * (T - 1) + d) return true;   // one within the other
  for (wide j = 1; j < H; ++j) {
    const wide i = j * b / a, rest = j * b - i * a;   // the tokens next to head j's start
    if ((i < T && rest < d) || (i + 1 < T && a - rest < d)) return false;
  }
  return true;
}

// Whether two gapless tensors [T][H][d] share memory. (Of tensors with gaps, slices of one buffer for instance,
// the ranges may cross although no element is in both; those are the caller's to keep apart.)
bool share_memory(const void* x, size_t x_bytes, const void* y, size_t y_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + y_bytes && b < a + x_bytes;
}
bool gapless(int T, int H, int d, long long tok, long long head) {
  return (T <= 1 || tok == (long long)H * d) && (H <= 1 || head == d);
}

bool rope_ok(const dllm_rope* r, int head_dim) {
  return r->rotary_dim >= 2 && r->rotary_dim % 2 == 0 && r->rotary_dim <= 2 * DLLM_ROPE_MAX_PAIRS &&
         r->rotary_dim <= head_dim && (r->layout == DLLM_ROPE_HALF || r->layout == DLLM_ROPE_INTERLEAVED);
}

RopeParams rope_params(const dllm_rope* r, bool transposed) {
  RopeParams p;
  p.rd = 0;
  p.interleaved = 0;
  p.sign = 1.f;
  p.mag = 1.0;
  if (!r) return p;
  p.rd = r->rotary_dim;
  p.interleaved = r->layout == DLLM_ROPE_INTERLEAVED;
  p.sign = transposed ? -1.f : 1.f;
  p.mag = r->magnitude;
  std::copy(r->turns, r->turns + p.rd / 2, p.turns);
  return p;
}

// 8-dim chunks lie on one side of the rotated part's borders.
bool rope_chunks(const dllm_rope* r) {
  return r->layout == DLLM_ROPE_INTERLEAVED ? r->rotary_dim % 8 == 0 : r->rotary_dim % 16 == 0;
}

bool cache_ok(const dllm_kv4* c) {
  return c && c->codes && c->scales && aligned16(c->codes) && aligned16(c->scales) && c->n_pages >= 1 &&
         c->page >= 16 && c->page <= 256 && (c->page & (c->page - 1)) == 0 && c->n_kv_heads >= 1 &&
         c->n_kv_heads <= 1024 && (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 176) &&
         (long long)c->n_pages * c->page <= 0x7FFFFFFFLL;
}

Kv4 cache_of(const dllm_kv4* c) {
  Kv4 k;
  k.codes = c->codes;
  k.scales = c->scales;
  k.n_pages = c->n_pages;
  k.page_shift = 0;
  while ((1 << k.page_shift) < c->page) ++k.page_shift;
  k.Hkv = c->n_kv_heads;
  k.hd = c->head_dim;
  return k;
}

bool addr_ok(const int32_t* req, const int32_t* pos, const int32_t* table, int n_req, int stride) {
  return req && pos && table && n_req >= 1 && stride >= 1;
}

// ---- attention: how a call is cut up

struct AttnPlan {
  int tiles, n_splits;
  int nr;    // 8-row columns of the few-row kernel; 0: the tensor-core kernel
  bool cut;  // which may cut tiles into parts
  int unit_shift;
};

// Few rows per KV head and request: the few-row kernel, 8 or 16 rows and a split of the keys per block.
// More: the tensor-core kernel, which deals its work out by itself.
AttnPlan attn_plan(int B, int T, int max_q, int max_kv, int group, int Hkv, int hd) {
  AttnPlan a{0, 1, 0, false, 0};
  const long rows = (long)max_q * group;
  // Two tiles of 16 rows unpack the cache twice, which at head_dim 64 and 128 is still faster than a tile of 256 rows
  // that is mostly empty: 32 rows of 8 KV heads over up to 4352 keys, 1, 8 and 64 requests, at head_dim 64 13, 31 and
  // 144 us against 19, 37 and 158, at 128 17, 42 and 204 against 21, 43 and 232, but at 176 22, 60 and 311 against 22,
  // 52 and 278; and 48 rows at head_dim 64 16, 40 and 184 against 19, 32 and 161.
  a.nr = rows <= 8 ? 1 : rows <= (hd == 176 ? 16 : 32) ? 2 : 0;
  if (a.nr == 0) {
    // what the requests' work adds up to stays below 2^31
    const long tiles = Hkv * std::min((long)B * ceil_div(rows, 256), (long)T * group / 256 + B);
    while (tiles * (8 + (ceil_div(max_kv, 48) >> a.unit_shift)) >= 0x7FFFFFFFL && a.unit_shift < 30) ++a.unit_shift;
    a.tiles = (int)std::min(tiles, 0x7FFFFFFFL);
    // Whether any lengths within the bounds can make the kernel find that cutting tiles pays, by 2 blocks of keys at
    // least: else the launch that joins parts (2 us) is left out. 36 requests of 64 queries over 128 keys at head_dim
    // 64 10.9 us without it, 12.9 with it.
    const long most = hd == 64 ? AttnKv4TcCfg<64>::START + ceil_div(max_kv, AttnKv4TcCfg<64>::BK)
                               : AttnKv4TcCfg<176>::START + ceil_div(max_kv, AttnKv4TcCfg<176>::BK);
    a.cut = ceil_div(tiles, kSMs) * most > kv4_cut_cost(kSMs, hd) + 2;
    return a;
  }
  a.tiles = ceil_div(rows, 8 * a.nr);
  // Blocks that the GPU holds at a time, and blocks without a split.
  const long slots = kSMs * (a.nr == 1   ? AttnKv4Cfg<64, 1>::BLOCKS
                             : hd == 176 ? AttnKv4Cfg<176, 2>::BLOCKS
                                         : AttnKv4Cfg<64, 2>::BLOCKS);
  const long blocks = (long)B * Hkv * a.tiles;
  long want;
  if (blocks * ceil_div(max_kv, 256) <= slots) {
    want = ceil_div(max_kv, 256);                      // a short call: as wide as it goes
  } else {
    // One wave of blocks if every tile has two splits or more in it: 24 tokens over up to 4352 keys (192 tiles of 8 KV
    // heads) 50 us in 3 splits, 57 in 7. Else about two waves, of 512 keys or more per block, so that requests of
    // different lengths even out: 64 tokens (512 tiles) 111 us in 3 splits, 116 in 1.
    want = 2 * blocks <= slots ? slots / blocks : std::min<long>(ceil_div(2 * slots, blocks), ceil_div(max_kv, 512));
  }
  want = std::max(1L, std::min<long>(want, ceil_div(max_kv, 64)));
  const int stage = 128;   // keys; no more splits than there are stages, or fill them
  a.n_splits = std::max(1, ceil_div(max_kv, std::max(stage, ceil_div(ceil_div(max_kv, want), stage) * stage)));
  return a;
}

size_t attn_workspace(const AttnPlan& a, int T, int H, int hd) {
  if (a.nr == 0) return !a.cut ? 0 : (size_t)kSMs * 2 * (256 * (hd + 1) * sizeof(float) + sizeof(int4));
  if (a.n_splits == 1) return 0;
  return (size_t)a.n_splits * T * H * (hd + 1) * sizeof(float);
}

bool attn_sizes_ok(const dllm_kv4* c, int B, int T, int max_q, int max_kv, int H) {
  return B >= 0 && B <= 65535 && T >= 0 && max_q >= 0 && max_q <= T && max_kv >= 0 && max_kv < (1 << 29) && H >= 1 &&
         H % c->n_kv_heads == 0 && H / c->n_kv_heads <= 128 && (long long)T * H <= 0x7FFFFFFFLL;
}

template <int HD, int NR>
cudaError_t run_few(cudaStream_t st, const AttnPlan& a, const AttnKv4Params& p) {
  using G = AttnKv4Cfg<HD, NR>;
  cudaError_t e = cudaSuccess;
  if (G::kTotal > 48 * 1024) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(attn_kv4_kernel<HD, NR>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, G::kTotal);
    if (e != cudaSuccess) return e;
  }
  return launch(st, attn_kv4_kernel<HD, NR>, dim3(a.n_splits, p.c.Hkv * a.tiles, p.B), G::THREADS, G::kTotal, p);
}

template <int HD>
cudaError_t run_tc(cudaStream_t st, const AttnPlan& a, const AttnKv4Params& p) {
  using G = AttnKv4TcCfg<HD>;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(attn_kv4_tc_kernel<HD>),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, G::kTotal);
  if (e != cudaSuccess) return e;
  return launch(st, attn_kv4_tc_kernel<HD>, dim3(kSMs), G::THREADS, G::kTotal, p);
}

template <int HD>
cudaError_t run_attn(cudaStream_t st, const AttnPlan& a, const AttnKv4Params& p) {
  cudaError_t e = a.nr == 1 ? run_few<HD, 1>(st, a, p) : a.nr == 2 ? run_few<HD, 2>(st, a, p) : run_tc<HD>(st, a, p);
  if (e != cudaSuccess) return e;
  if (a.nr == 0) return !a.cut ? e : launch(st, attn_kv4_parts_kernel<HD>, dim3(4 * kSMs), 256, 0, p, kSMs);
  if (a.n_splits > 1) e = launch(st, attn_kv4_merge_kernel<HD>, dim3((unsigned)p.max_q * p.H, p.B), 128, 0, p);
  return e;
}

template <typename TI, typename TO>
cudaError_t run_rope(cudaStream_t st, bool vec, const RopeParams& r, const void* x, long xt, long xh, const int32_t* pos,
                     int T, int H, int hd, void* y, long yt, long yh) {
  const int rot_units = vec ? (r.interleaved ? r.rd / 8 : r.rd / 16) : r.rd / 2;
  const int head_units = rot_units + (hd - r.rd) / (vec ? 8 : 1);
  int threads;
  const TokenTiling tl = token_tiling(H * head_units, T, r.rd, kSMs, &threads);
  auto kern = vec ? rope_kernel<TI, TO, true> : rope_kernel<TI, TO, false>;
  return launch(st, kern, dim3(ceil_div(T, tl.tb)), threads, sizeof(float4) * tl.tb * rope_stride(r.rd), r,
                reinterpret_cast<const TI*>(x), xt, xh, pos, T, head_units, rot_units, reinterpret_cast<TO*>(y), yt, yh,
                tl);
}

template <int HD, typename TI>
cudaError_t run_append_hd(cudaStream_t st, bool vec, const RopeParams& r, const Kv4& c, const Kv4Addr& a, const void* k,
                          long kt, long kh, const void* v, long vt, long vh, const int32_t* rope_pos, int T) {
  int threads;
  const TokenTiling tl = token_tiling(2 * c.Hkv * (HD / 8), T, r.rd, kSMs, &threads);
  auto kern = vec ? kv4_append_kernel<HD, TI, true> : kv4_append_kernel<HD, TI, false>;
  return launch(st, kern, dim3(ceil_div(T, tl.tb)), threads, sizeof(float4) * tl.tb * rope_stride(r.rd), r, c, a,
                reinterpret_cast<const TI*>(k), kt, kh, reinterpret_cast<const TI*>(v), vt, vh, rope_pos, T, tl);
}

template <typename TI>
cudaError_t run_append(cudaStream_t st, bool vec, const RopeParams& r, const Kv4& c, const Kv4Addr& a, const void* k,
                       long kt, long kh, const void* v, long vt, long vh, const int32_t* rope_pos, int T) {
  auto f = c.hd == 176 ? run_append_hd<176, TI> : c.hd == 128 ? run_append_hd<128, TI> : run_append_hd<64, TI>;
  return f(st, vec, r, c, a, k, kt, kh, v, vt, vh, rope_pos, T);
}

}  // namespace

extern "C" {

int dllm_rope_init(dllm_rope* out, int rotary_dim, int layout, double theta, int scaling, double factor,
                   double original_ctx, double beta_fast, double beta_slow) {
  if (!out || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 2 * DLLM_ROPE_MAX_PAIRS ||
      (layout != DLLM_ROPE_HALF && layout != DLLM_ROPE_INTERLEAVED) || !(theta > 1.0) || !std::isfinite(theta) ||
      scaling < DLLM_ROPE_NONE || scaling > DLLM_ROPE_YARN)
    return DLLM_E_INVAL;
  if (scaling != DLLM_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return DLLM_E_INVAL;
  if (scaling == DLLM_ROPE_NTK && rotary_dim < 4) return DLLM_E_INVAL;
  if (scaling == DLLM_ROPE_YARN && (!(original_ctx >= 1.0) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
                                    !std::isfinite(original_ctx) || !std::isfinite(beta_fast)))
    return DLLM_E_INVAL;
  const double two_pi = 6.283185307179586476925286766559;
  const double rd = rotary_dim;
  out->rotary_dim = rotary_dim;
  out->layout = layout;
  out->magnitude = 1.0;
  double base = theta;
  if (scaling == DLLM_ROPE_NTK) base = theta * std::pow(factor, rd / (rd - 2.0));
  double low = 0.0, high = 0.0;
  if (scaling == DLLM_ROPE_YARN) {
    // the pair that turns `beta` times over the original context, as a real index
    auto at = [&](double beta) { return rd * std::log(original_ctx / (beta * two_pi)) / (2.0 * std::log(theta)); };
    low = std::max(std::floor(at(beta_fast)), 0.0);
    high = std::min(std::ceil(at(beta_slow)), rd - 1.0);
    out->magnitude = 0.1 * std::log(factor) + 1.0;
  }
  for (int i = 0; i < DLLM_ROPE_MAX_PAIRS; ++i) {
    double f = 0.0;
    if (i < rotary_dim / 2) {
      f = std::pow(base, -2.0 * i / rd);
      if (scaling == DLLM_ROPE_LINEAR) f /= factor;
      if (scaling == DLLM_ROPE_YARN) {
        const double ramp = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
        f = f * (1.0 - ramp) + f / factor * ramp;
      }
    }
    out->turns[i] = f / two_pi;
  }
  return DLLM_OK;
}

int dllm_op_rope(const dllm_rope* rope, const void* x, int x_type, long long x_token_stride, long long x_head_stride,
                 const int32_t* pos, int T, int H, int head_dim, void* y, int y_type, long long y_token_stride,
                 long long y_head_stride, int transposed, void* stream) {
  if (!rope || (x_type != DLLM_F32 && x_type != DLLM_BF16) || (y_type != DLLM_F32 && y_type != DLLM_BF16) || T < 0 ||
      H < 1 || H > 32768 || head_dim < 2 || head_dim > 1024 || (long)H * head_dim > (1 << 20) || !rope_ok(rope, head_dim))
    return DLLM_E_INVAL;
  if (T == 0) return DLLM_OK;
  if (!x || !y || !pos) return DLLM_E_INVAL;
  if (x == y && (x_type != y_type || x_token_stride != y_token_stride || x_head_stride != y_head_stride))
    return DLLM_E_INVAL;
  if (!rows_apart(T, H, head_dim, y_token_stride, y_head_stride)) return DLLM_E_INVAL;
  const size_t n = (size_t)T * H * head_dim;
  if (x != y && gapless(T, H, head_dim, x_token_stride, x_head_stride) &&
      gapless(T, H, head_dim, y_token_stride, y_head_stride) && share_memory(x, n * size_of(x_type), y, n * size_of(y_type)))
    return DLLM_E_INVAL;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const RopeParams r = rope_params(rope, transposed != 0);
  const bool vec = vectors(x, x_type, x_token_stride, x_head_stride) &&
                   vectors(y, y_type, y_token_stride, y_head_stride) && rope_chunks(rope) && head_dim % 8 == 0;
  auto f = x_type == DLLM_F32 ? (y_type == DLLM_F32 ? run_rope<float, float> : run_rope<float, bf16_t>)
                              : (y_type == DLLM_F32 ? run_rope<bf16_t, float> : run_rope<bf16_t, bf16_t>);
  return status(f(st, vec, r, x, x_token_stride, x_head_stride, pos, T, H, head_dim, y, y_token_stride, y_head_stride));
}

int dllm_op_append_kv4(const dllm_kv4* cache, const void* k, long long k_token_stride, long long k_head_stride,
                       const void* v, long long v_token_stride, long long v_head_stride, int type, const int32_t* req,
                       const int32_t* pos, const int32_t* rope_pos, int T, const int32_t* table, int n_req,
                       int table_stride, const dllm_rope* rope, void* stream) {
  if (!cache_ok(cache) || (type != DLLM_F32 && type != DLLM_BF16) || T < 0 || (rope && !rope_ok(rope, cache->head_dim)))
    return DLLM_E_INVAL;
  if (T == 0) return DLLM_OK;
  if (!k || !v || !addr_ok(req, pos, table, n_req, table_stride)) return DLLM_E_INVAL;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const RopeParams r = rope_params(rope, false);
  const bool vec = vectors(k, type, k_token_stride, k_head_stride) && vectors(v, type, v_token_stride, v_head_stride) &&
                   (!rope || rope_chunks(rope));
  const Kv4Addr a{req, pos, table, n_req, table_stride};
  auto f = type == DLLM_F32 ? run_append<float> : run_append<bf16_t>;
  return status(f(st, vec, r, cache_of(cache), a, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride,
                  rope_pos ? rope_pos : pos, T));
}

int dllm_op_read_kv4(const dllm_kv4* cache, const int32_t* req, const int32_t* pos, int T, const int32_t* table,
                     int n_req, int table_stride, uint16_t* k_out, uint16_t* v_out, int zero_padding, void* stream) {
  if (!cache_ok(cache) || T < 0 || !aligned16(k_out) || !aligned16(v_out)) return DLLM_E_INVAL;
  if (T == 0 || (!k_out && !v_out)) return DLLM_OK;
  const size_t bytes = (size_t)T * cache->n_kv_heads * cache->head_dim * 2;
  if (k_out && v_out && share_memory(k_out, bytes, v_out, bytes)) return DLLM_E_INVAL;
  if (!addr_ok(req, pos, table, n_req, table_stride)) return DLLM_E_INVAL;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Kv4Addr a{req, pos, table, n_req, table_stride};
  auto kern = cache->head_dim == 176   ? kv4_read_kernel<176>
              : cache->head_dim == 128 ? kv4_read_kernel<128>
                                       : kv4_read_kernel<64>;
  return status(launch(st, kern, dim3(ceil_div(T, 8)), 256, 0, cache_of(cache), a, T, k_out, v_out, zero_padding));
}

long long dllm_op_attn_kv4_workspace(const dllm_kv4* cache, int B, int T, int max_q, int max_kv, int H) {
  if (!cache_ok(cache) || !attn_sizes_ok(cache, B, T, max_q, max_kv, H)) return DLLM_E_INVAL;
  if (B == 0 || max_q == 0) return 0;
  const AttnPlan a = attn_plan(B, T, max_q, max_kv, H / cache->n_kv_heads, cache->n_kv_heads, cache->head_dim);
  return (long long)attn_workspace(a, T, H, cache->head_dim);
}

int dllm_op_attn_kv4(const dllm_kv4* cache, const uint16_t* q, long long q_token_stride, long long q_head_stride,
                     uint16_t* out, long long out_token_stride, long long out_head_stride, float* lse,
                     const int32_t* q_start, const int32_t* kv_len, int B, int T, int max_q, int max_kv, int H,
                     const int32_t* table, int table_stride, int causal, float scale, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!cache_ok(cache) || !attn_sizes_ok(cache, B, T, max_q, max_kv, H) || !(scale > 0.f) || !std::isfinite(scale))
    return DLLM_E_INVAL;
  if (B == 0 || max_q == 0) return DLLM_OK;
  if (!q || !out || !q_start || !kv_len || !table || table_stride < 1 ||
      !vectors(q, DLLM_BF16, q_token_stride, q_head_stride) ||
      !vectors(out, DLLM_BF16, out_token_stride, out_head_stride) || !aligned16(workspace))
    return DLLM_E_INVAL;
  if (!rows_apart(T, H, cache->head_dim, out_token_stride, out_head_stride)) return DLLM_E_INVAL;
  if (q == out ? (T > 1 && q_token_stride != out_token_stride) || (H > 1 && q_head_stride != out_head_stride)
               : gapless(T, H, cache->head_dim, q_token_stride, q_head_stride) &&
                     gapless(T, H, cache->head_dim, out_token_stride, out_head_stride) &&
                     share_memory(q, (size_t)T * H * cache->head_dim * 2, out, (size_t)T * H * cache->head_dim * 2))
    return DLLM_E_INVAL;
  const int group = H / cache->n_kv_heads;
  const AttnPlan a = attn_plan(B, T, max_q, max_kv, group, cache->n_kv_heads, cache->head_dim);
  // the few-row kernel's grid; the tensor-core kernel's sums
  if (a.nr ? (long)cache->n_kv_heads * a.tiles > 65535 : a.tiles > (1 << 27)) return DLLM_E_INVAL;
  if (attn_workspace(a, T, H, cache->head_dim) > (workspace ? workspace_bytes : 0)) return DLLM_E_INVAL;
  AttnKv4Params p;
  p.c = cache_of(cache);
  p.q = q;
  p.q_tok = q_token_stride;
  p.q_head = q_head_stride;
  p.out = out;
  p.o_tok = out_token_stride;
  p.o_head = out_head_stride;
  p.lse = lse;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.table = table;
  p.stride = table_stride;
  p.B = B;
  p.T = T;
  p.H = H;
  p.group = group;
  p.max_q = max_q;
  p.max_kv = max_kv;
  p.causal = causal != 0;
  p.n_splits = a.n_splits;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.mask_low = 0x003C003Cu;
  p.mask_high = 0x03C003C0u;
  p.mask_bf16 = 0x00780078u;
  p.part_o = reinterpret_cast<float*>(workspace);
  const size_t part_rows = a.nr == 0 ? (size_t)kSMs * 512 : (size_t)a.n_splits * T * H;
  p.part_lse = p.part_o + part_rows * cache->head_dim;
  p.cut = a.cut;
  p.unit_shift = a.unit_shift;
  p.parts = reinterpret_cast<int4*>(p.part_lse + part_rows);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->head_dim == 176   ? run_attn<176>(st, a, p)
                        : cache->head_dim == 128 ? run_attn<128>(st, a, p)
                                                 : run_attn<64>(st, a, p);
  return status(e);
}

}  // extern "C"

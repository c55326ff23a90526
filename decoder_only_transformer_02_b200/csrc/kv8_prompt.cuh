// Attention of many new tokens per sequence over the paged 8-bit cache (the
// chunks of a prompt), on the 5th-generation tensor cores.
//
// The rows of one sequence and key/value head, (token, head of the group)
// pairs, are taken 256 at a time, as two tiles of 128 that share every key and
// value block of 128 tokens:
//   S_j = Q K_j^T     tcgen05.mma, M = 128, N = 128 keys, K = d, f16 in, fp32 in TMEM
//   P_j = 2^(S_j f - m + 6) in f16, back into TMEM   (one thread per row)
//   O  += P_j V_j     A = P_j from TMEM, N = d, K = 128 keys
// and the result is O / sum P as in the streaming kernel (kv8_attention.cuh).
//
// The tensor cores read f16 from shared memory, the cache holds 8-bit codes, so
// six warps convert each block on its way: the codes of the next 16 KB are
// loaded while these 16 KB are converted and stored as swizzled f16 tiles.  A
// key block's values are code * scale / (the block's largest scale), exact in
// f16 up to a ratio of 2^24 (int8) or 2^15 (e4m3); the largest scale multiplies
// the scores.  Values are taken relative to the largest scale so far; when that
// rises, O is scaled down as it is when the row maximum moves.
// A block whose pages' scales may lie further apart is stored as bare codes.  The
// softmax then multiplies a page's scores by its scale, and its weights by its
// value scale over the largest that the row sees: what a row does not see, or
// gives no weight, must not take the precision of what it does (far_block).
//
// Roles (512 threads of 128 registers, one CTA per SM): warps 0-3, 14 and 15
// convert, warps 4-7 and 8-11 are the softmax of tile 0 and 1, warps 12 and 13
// issue their MMAs.  Two tiles per CTA instead of two CTAs of one tile: the
// conversion is done once for both, and one tile's exponentials run while the
// other's MMAs do.  (Registers moved from the converting warps to the softmax
// cost more there than they gave here.)
//
// As in the streaming kernel the key blocks of all items are one line of work
// cut into equal parts, one per SM, and the cut items are joined by a second
// kernel: four chunks of 300 to 1024 rows are 120 items of unequal length, which
// taken whole would leave SMs idle and others twice as busy.
//
// Measured: 64 sequences of 256 new tokens over 4096, 12 heads: 443 us at d = 64
// (451 TFLOP/s), 683 at d = 128 (585); one tile per item (128 new tokens) 356 us;
// four chunks of 300 to 1024 over 1500 to 4096: 62 us.  The softmax warps'
// chain from TMEM load to store bounds it (MUFU 45% busy, tensor pipe 22%), and at
// d = 128 the conversion.  With 128 registers a thread, 22 words are spilled and
// 53 (63) read back.
//
// All waits are bounded.
#pragma once
#include "attention_tc.cuh"
#include "kv8_attention.cuh"

namespace kv8 {

constexpr int W_THREADS = 512;
constexpr int W_CONV = 6;    // converting warps
constexpr int W_ROWS = 256;  // rows of a work item (two tiles)
constexpr int W_KEYS = 128;  // keys of a block

template <int D>
struct Wide {
  static constexpr int NS = D == 64 ? 4 : 2;             // stages of the key/value ring
  static constexpr int TILE = 128 * D * 2;               // one f16 tile: Q, K or V
  static constexpr int KV_OFF = 2 * TILE;                // after the two Q tiles; stage s: K, V
  static constexpr int BAR_OFF = KV_OFF + NS * 2 * TILE;
  static constexpr int INFO_OFF = BAR_OFF + 256;         // float2 per stage: key block scale (< 0: apart), value scale so far
  static constexpr int APART_OFF = INFO_OFF + 256;       // float2 per stage and page of the block: key and value scale
  static constexpr int LINE_OFF = APART_OFF + 256;
  static constexpr int UNITS = D / 64;                   // 16 KB units of codes in a block: all of it, or keys, values
  // TMEM columns of a tile: S, P (in place of S's first 64 when d = 128), O
  static constexpr uint32_t T_P = D == 64 ? 128 : 0, T_O = D == 64 ? 192 : 128;
  static size_t bytes(int n) { return LINE_OFF + (size_t)(n + 1) * 8 + 1024; }
};

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// f16 instruction descriptor: fp32 accumulate, M = 128; A K-major, B K-major or MN-major
__host__ __device__ constexpr uint32_t f16_idesc(int n, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// V as B operand: rows of 128 bytes (64 dimensions), one per key; the second 64 dimensions 16 KB on
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(16384u >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// ------------------------------------------------------------- the work line
// Item j of a sequence (rows 256 j ..) and head takes the blocks up to its
// last row's token, and `setup` units more.
__device__ __forceinline__ int item_blocks(const Call& k, int len, int q, int j) {
  const int last = min(q * k.group, (j + 1) * W_ROWS) - 1;
  return (len - q + last / k.group) / W_KEYS + 1;
}
__device__ __forceinline__ int items_of(const Call& k, int q) { return (q * k.group + W_ROWS - 1) / W_ROWS; }

// what a block counts: with two tiles a third more than with one (2.6 and 2.0 us)
__device__ __forceinline__ int item_cost(const Call& k, int q, int j) { return q * k.group - j * W_ROWS > 128 ? 4 : 3; }

__device__ __forceinline__ bool lay_out_wide(const Call& k, long long* pre, long long* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const bool report = blockIdx.x == 0;
  long long base = 0;
  bool bad = false;
  for (int i0 = 0; i0 < k.n; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    long long x = 0;
    if (i < k.n) {
      const int a = k.cu[i], b = k.cu[i + 1], q = b - a;
      bad |= a < 0 || b < a || b > k.rows;
      if (q > 0 && (long)q * k.group > k.narrow) {
        const int len = k.c.len_of(k.slots[i]);
        if (len < q || q > k.max_q) {
          if (report) set_device_err(DERR_KV8_ARGS);
        } else if (b <= k.rows) {
          const int items = items_of(k, q);
          for (int j = 0; j < items; ++j) x += item_blocks(k, len, q, j) * item_cost(k, q, j) + k.setup;
          x *= k.c.kvh;
        }
      }
    }
    const long long own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long before = base;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += s_warp[w];
      base += s_warp[w];
    }
    if (i < k.n) pre[i] = before + x - own;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[k.n] = base;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && report) set_device_err(DERR_KV8_ARGS);
    return false;
  }
  return true;
}

struct Item {
  int slot, len, a, q, head, row0;  // row0: first of its rows
  int b0, b1, blocks;               // blocks [b0, b1) of `blocks` are this part's
  long long next;
  int left;                         // units of it behind this part
};
__device__ __forceinline__ Item item_at(const Call& k, const long long* pre, long long at, long long end) {
  int lo = 0, hi = k.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= at) lo = mid; else hi = mid;
  }
  Item p;
  p.slot = k.slots[lo];
  p.len = k.c.lens[p.slot];
  p.a = k.cu[lo];
  p.q = k.cu[lo + 1] - p.a;
  long long rel = at - pre[lo];
  int j = 0, size, cost;
  for (;; ++j) {  // head after head within an item's rows
    p.blocks = item_blocks(k, p.len, p.q, j);
    cost = item_cost(k, p.q, j);
    size = p.blocks * cost + k.setup;
    if (rel < (long long)size * k.c.kvh) break;
    rel -= (long long)size * k.c.kvh;
  }
  p.head = (int)(rel / size);
  p.row0 = j * W_ROWS;
  const int u = (int)(rel - (long long)p.head * size);
  p.next = min(at - u + size, end);
  p.b0 = max(0, u - k.setup) / cost;
  p.b1 = max(0, (int)(p.next - at) + u - k.setup) / cost;
  p.left = (int)(at - u + size - p.next);
  return p;
}

// sixteen codes to f16 times a power of two (as a pair in f)
template <int FMT>
__device__ __forceinline__ void codes16_half(uint4 w, uint32_t f, uint32_t (&h)[8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  if (FMT == GPT2_KV_E4M3) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * i]) : "r"(e4m3x2_to_half2(x[i] & 0xffffu)), "r"(f));
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * i + 1]) : "r"(e4m3x2_to_half2(x[i] >> 16)), "r"(f));
    }
  } else {
    uint32_t n;  // -1152 f
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(n) : "r"(f), "r"(0xE480E480u));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = x[i] ^ 0x80808080u;  // code + 128, under the exponent of 1024
      const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[2 * i]) : "r"(a), "r"(f), "r"(n));
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[2 * i + 1]) : "r"(b), "r"(f), "r"(n));
    }
  }
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The softmax of a block whose pages' scales may lie apart (scale.x < 0), or whose
// scores may pass 2^20 (a sum of products is below 2^30): there the fused z of the
// common case would differ from the maximum, which is rounded, by half their last
// place.  Rare, so the loop over the blocks is left for it and entered again: as a
// branch in the loop it made the common case slower by a tenth (of which 3% are
// left: 64 sequences of 256 over 4096 427 -> 442 us, one tile per item 346 -> 356,
// four chunks 61.7 -> 62.4; nothing at d = 128).
template <int D>
__device__ __noinline__ void far_rescale(uint32_t tl, float f) {  // the row's O
  tcg::tc_fence_after();
#pragma unroll 1
  for (int q = 0; q < D / 8; ++q) {
    uint32_t o[8];
    tmem_ld8(tl + Wide<D>::T_O + 8 * q, o);
    tcg::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
    tmem_st8(tl + Wide<D>::T_O + 8 * q, o);
  }
  tcfa::tmem_wait_st();
  tcg::tc_fence_before();
}
struct FarRow {
  float m, l, vref, rowf;
};
template <int D>
__device__ __noinline__ bool far_block(FarRow& row, uint32_t tl, float2 scale, const volatile float2* pages, int ps_log2,
                                       int last, uint64_t* pv_done, uint32_t phase) {
  const bool apart = scale.x < 0.f;
  float m = row.m, l = row.l, vref = row.vref, alpha = 1.f;
  float vtop = apart ? vref : scale.y, mx = -INFINITY;
  auto factor = [&](int i) { return fmaxf((apart ? pages[i * 16 >> ps_log2].x : scale.x) * row.rowf, 1e-37f); };  // of 16 tokens' scores
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    uint32_t v[16];
    tcg::tmem_ld16(tl + 16 * i, v);
    const float f = factor(i);
    if (apart && 16 * i <= last) vtop = fmaxf(vtop, pages[i * 16 >> ps_log2].y);
    tcg::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, 16 * i + e > last ? -INFINITY : __uint_as_float(v[e]) * f);
  }
  const bool moved = __any_sync(0xffffffffu, mx > m + 8.f);
  const bool rescale = __any_sync(0xffffffffu, moved || vtop > vref);
  if (moved) {
    const float nm = fmaxf(m, mx);
    alpha = m == -INFINITY ? 0.f : ex2_approx(m - nm);
    m = nm;
    l *= alpha;
  }
  if (vtop > vref) {
    alpha *= vref / vtop;
    vref = vtop;
  }
  const float off = m == -INFINITY ? 0.f : m - 6.f, vinv = vref > 0.f ? 1.f / vref : 0.f;
  if (pv_done && !tcfa::warp_wait(pv_done, phase)) return false;
  tcg::tc_fence_after();
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {  // (P's columns lie at or before those of the scores)
    uint32_t v[16], y[8];
    tcg::tmem_ld16(tl + 16 * i, v);
    // a page that the row does not see may have a larger scale, but its weights are 0
    const float f = factor(i), w = apart ? fminf(pages[i * 16 >> ps_log2].y * vinv, 1.f) : 1.f;
    tcg::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float z0 = 16 * i + e > last ? 0.f : ex2_approx(__fmul_rn(__uint_as_float(v[e]), f) - off);
      const float z1 = 16 * i + e + 1 > last ? 0.f : ex2_approx(__fmul_rn(__uint_as_float(v[e + 1]), f) - off);
      l += z0 + z1;
      y[e >> 1] = half2_of(z0 * w, z1 * w);
    }
    tmem_st8(tl + Wide<D>::T_P + 8 * i, y);
  }
  if (pv_done && rescale) far_rescale<D>(tl, alpha);
  tcfa::tmem_wait_st();
  tcg::tc_fence_before();
  __syncwarp();
  row.m = m, row.l = l, row.vref = vref;
  return true;
}

template <int FMT, int D>
__global__ void __launch_bounds__(W_THREADS, 1) wide_kernel(const Call k) {
  using S = Wide<D>;
  using namespace tcg;
  using namespace tcfa;
  constexpr int NS = S::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);  // NS, count W_CONV
  uint64_t* kv_empty = kv_full + NS;                                   // NS, count 2: the tile's MMAs have read the stage
  uint64_t* q_full = kv_empty + NS;                                    // 2, count 4: the tile's Q is in shared memory
  uint64_t* s_full = q_full + 2;                                       // 2: S in TMEM
  uint64_t* s_free = s_full + 2;                                       // 2, count 4: S is in registers
  uint64_t* p_full = s_free + 2;                                       // 2, count 4: P in TMEM (and O rescaled)
  uint64_t* pv_done = p_full + 2;                                      // 2: O += P V complete
  uint64_t* drain = pv_done + 2;                                       // 2
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  float2* info = reinterpret_cast<float2*>(smem + S::INFO_OFF);
  float2* apart_at = reinterpret_cast<float2*>(smem + S::APART_OFF);
  long long* s_warp = reinterpret_cast<long long*>(smem + S::INFO_OFF + 128);
  long long* pre = reinterpret_cast<long long*>(smem + S::LINE_OFF);
  const Cache& c = k.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch();
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], W_CONV);
      mbar_init(&kv_empty[s], 2);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&q_full[a], 4);
      mbar_init(&s_full[a], 1);
      mbar_init(&s_free[a], 4);
      mbar_init(&p_full[a], 4);
      mbar_init(&pv_done[a], 1);
      mbar_init(&drain[a], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const bool line_ok = lay_out_wide(k, pre, s_warp);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long total = line_ok ? pre[k.n] : 0;
  const long long per = max((long long)k.min_part, (total + gridDim.x - 1) / gridDim.x);
  long long at = blockIdx.x * per;
  const long long end = min(total, at + per);

  if (warp == 12 || warp == 13) {
    if (lane == 0) {
      // ---------------------------------------------- MMA issuer of a tile
      const int a = warp - 12;
      constexpr uint32_t id_s = f16_idesc(W_KEYS, 0), id_pv = f16_idesc(D, 1);
      const uint32_t qa = smem_u32(smem + a * S::TILE), ta = tmem + a * 256;
      uint32_t g = 0, t = 0, items = 0;
      bool ok = true;
      int join_parts = 0;
      auto do_pv = [&](uint32_t gp, bool first) {  // of the tile's latest S, whose block is number gp
        if (!mbar_wait(&p_full[a], (t - 1) & 1u)) return false;
        tc_fence_after();
        const uint32_t va = smem_u32(smem + S::KV_OFF + (2 * (gp % NS) + 1) * S::TILE);
#pragma unroll
        for (int kk = 0; kk < W_KEYS / 16; ++kk)
          tc_mma_ts(ta + S::T_O, ta + S::T_P + kk * 8, v_desc(va + kk * 2048), id_pv, first && kk == 0 ? 0u : 1u);
        tc_commit(&pv_done[a]);
        tc_commit(&kv_empty[gp % NS]);
        return true;
      };
      while (ok && at < end) {
        const Item p = item_at(k, pre, at, end);
        const int rows = p.q * k.group - p.row0;
        if (a == 0 && p.b0 == 0 && p.b1 > 0 && p.b1 < p.blocks) {
          join_parts = (int)((p.next + p.left - 1) / per) - blockIdx.x + 1;
          Join j;
          j.parts = join_parts, j.tile_rows = min(W_ROWS, rows), j.row0 = p.row0, j.head = p.head, j.a = p.a;
          k.join[blockIdx.x] = j;
        }
        at = p.next;
        if (rows <= a * 128) {  // only the other tile has rows: let go of its blocks as they come
          for (int j = p.b0; ok && j < p.b1; ++j, ++g) {
            ok = mbar_wait(&kv_full[g % NS], (g / NS) & 1u);
            if (ok) mbar_arrive(&kv_empty[g % NS]);
          }
          continue;
        }
        for (int j = p.b0; ok && j < p.b1; ++j, ++g, ++t) {
          const int s = g % NS;
          if (j == p.b0) {
            ok = mbar_wait(&q_full[a], items & 1u);
            ++items;
          } else if (D == 64) {
            ok = mbar_wait(&s_free[a], (t - 1) & 1u);
          } else {
            ok = do_pv(g - 1, j - 1 == p.b0);  // P lies in S's place: its product goes first
          }
          ok = ok && mbar_wait(&kv_full[s], (g / NS) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ka = smem_u32(smem + S::KV_OFF + 2 * s * S::TILE);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
            tc_mma(ta, make_sdesc(qa + o, 0), make_sdesc(ka + o, 0), id_s, kk > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[a]);
          if (D == 64 && j > p.b0) ok = do_pv(g - 1, j - 1 == p.b0);
        }
        if (ok && p.b1 > p.b0) ok = do_pv(g - 1, p.b1 - 1 == p.b0);
      }
      if (a == 0 && join_parts == 0) k.join[blockIdx.x].parts = 0;
      if (!ok) set_device_err(DERR_WAIT_TIMEOUT);
      tc_commit(&drain[a]);
      if (!mbar_wait_drain(&drain[a], 0)) set_device_err(DERR_WAIT_TIMEOUT);
    }
  } else if (warp < 4 || warp > 13) {
      // ------------------------------------------------ converting warps
      // A unit is 32 pieces of 512 bytes: 512 / D consecutive tokens' codes, 16
      // bytes for each lane; warp w takes the pieces w, w + 6, ...
      constexpr int ROWS = 512 / D, PER_SIDE = W_KEYS / ROWS, NX = (32 + W_CONV - 1) / W_CONV;
      const int cw = warp < 4 ? warp : warp - 10;
      // a lane's row and 16-byte piece in it: every eight lanes hold two rows of four
      // pieces, whose f16 values the swizzle puts into different banks
      const int lrow = D == 64 ? lane >> 2 : (lane >> 2) & 3, lq = D == 64 ? lane & 3 : (lane & 3) + 4 * (lane >> 4);
      auto mine = [&](int e) { return cw + W_CONV * e < 32; };
      // where the lane's two f16 pieces go within eight rows (the row among them is the same for all of a warp's pieces)
      static_assert(W_CONV % 2 == 0, "pieces of four rows keep their place among eight");
      const int row7 = D == 64 ? lrow : (cw & 1) * 4 + lrow;
      const uint32_t lane_to = row7 * 128 + (((2 * lq & 7) ^ row7) << 4) + (lq >> 2) * 16384;
      const int lane_from = lrow * D + lq * 16;
      uint32_t g = 0;
      bool ok = true;
      const long page_stride = c.page_bytes();
      const long side_stride = (long)c.kvh * c.ps * D;
      while (ok && at < end) {
        const Item p = item_at(k, pre, at, end);
        at = p.next;
        if (p.b1 == p.b0) continue;
        const int32_t* table = c.table + (long)p.slot * c.max_pages;
        const uint8_t* head_base = c.codes + ((long)k.layer * 2 * c.kvh + p.head) * c.ps * D;
        const int per_block = W_KEYS >> c.ps_log2;  // pages of a block
        // Loads run a block ahead: the codes of block j + 1, the scales of its
        // pages and the page ids of block j + 2 are requested before block j
        // is converted.  The processor counts a warp's open loads in a few
        // counters that it shares among them, so waiting for an old load may
        // wait for a new one: `after` makes every new address depend on what
        // the old loads brought (by a zero that the compiler does not know).
        // What lies behind the last token is read (of its last page) and
        // cleared before it is converted.
        const int last_page = c.pages_of(p.len) - 1;
        auto page_id = [&](int blk) {  // lane x: page x of the block
          return table[min(blk * per_block + min(lane, per_block - 1), last_page)];
        };
        auto valid = [&](int page) { return c.page_ok(page) ? page : 0; };
        uint4 nx[NX] = {};
        auto load = [&](int page, int unit, uint32_t after) {  // the warp's pieces of a unit
#pragma unroll
          for (int e = 0; e < NX; ++e)
            if (mine(e)) {
              const int i = cw + W_CONV * e + 32 * unit, row0 = (i & (PER_SIDE - 1)) * ROWS;
              const int pg = __shfl_sync(0xffffffffu, page, row0 >> c.ps_log2);
              nx[e] = __ldcg(reinterpret_cast<const uint4*>(head_base + pg * page_stride + (i >= PER_SIDE ? side_stride : 0) +
                                                            ((row0 & (c.ps - 1)) * D + lane_from + after)));
            }
        };
        float vref = 0.f;
        int page = page_id(p.b0), page1 = page_id(p.b0 + 1);
        bool bad = !c.page_ok(page);
        page = valid(page);
        float ks = c.scales[c.unit(page, k.layer, 0, p.head)], vs = c.scales[c.unit(page, k.layer, 1, p.head)];
        uint32_t kexp = __shfl_sync(0xffffffffu, __float_as_uint(ks) >> 23, 0), vexp = __shfl_sync(0xffffffffu, __float_as_uint(vs) >> 23, 0);
        load(page, 0, 0);
        for (int j = p.b0; j < p.b1; ++j, ++g) {
          const int s = g % NS;
          // factors of the block's pages
          if (bad) set_device_err(DERR_KV8_TABLE);
          const uint32_t bads = __ballot_sync(0xffffffffu, bad);  // pages whose codes are not the sequence's
          const bool nan = bad || !(ks <= 3.0e38f && vs <= 3.0e38f);
          // apart: some scale more than half the exact range from what the blocks before had (so that the vote waits
          // for no reduction)
          constexpr int HALF = FMT == GPT2_KV_INT8 ? 12 : 7;
          const uint32_t kd = (__float_as_uint(ks) >> 23) - kexp + HALF, vd = (__float_as_uint(vs) >> 23) - vexp + HALF;
          const bool apart = __any_sync(0xffffffffu, !nan && max(kd, vd) > 2 * HALF);
          const float kmax = __uint_as_float(max(1u << 23, __reduce_max_sync(0xffffffffu, nan ? 0u : __float_as_uint(fabsf(ks)))));
          const float vmax = __uint_as_float(max(1u << 23, __reduce_max_sync(0xffffffffu, nan ? 0u : __float_as_uint(fabsf(vs)))));
          vref = fmaxf(vref, vmax);
          kexp = __float_as_uint(kmax) >> 23, vexp = __float_as_uint(vmax) >> 23;
          // (the conversion waits for this: divisions in place of the powers' inverses make 442 us 447, one tile 356 372)
          const float kr = apart ? 1.f : ks * inverse_pow2(__float_as_uint(kmax)), vr = apart ? 1.f : vs * inverse_pow2(__float_as_uint(vref));
          // a page with a scale that is not a number: its keys are not, its values 0 (only rows that see it notice)
          const uint32_t kf = nan ? 0x7e007e00u : half2_of(kr, kr), vf = nan ? 0u : half2_of(vr, vr);
          if (!__all_sync(0xffffffffu, mbar_wait(&kv_empty[s], ((g / NS) & 1u) ^ 1u))) {
            ok = false;
            break;
          }
          if (cw == 0 && lane == 0) info[s] = make_float2(apart ? -kmax : kmax, vref);
          if (apart && cw == 0 && lane < 8) apart_at[s * 8 + lane] = nan ? make_float2(0.f, 0.f) : make_float2(ks, vs);
          const int left = p.len - j * W_KEYS;  // tokens from the block on
#pragma unroll
          for (int u = 0; u < S::UNITS; ++u) {
            uint4 cur[NX];
            uint32_t after = page1 | kf | vf;
#pragma unroll
            for (int e = 0; e < NX; ++e) {
              cur[e] = nx[e];
              after |= cur[e].x | cur[e].y | cur[e].z | cur[e].w;
            }
            after &= k.zero;
            if (u + 1 < S::UNITS) {
              load(page, u + 1, after);
            } else if (j + 1 < p.b1) {
              bad = !c.page_ok(page1);
              page = valid(page1);
              load(page, 0, after);
              ks = c.scales[c.unit(page, k.layer, 0, p.head)];
              vs = c.scales[c.unit(page, k.layer, 1, p.head)];
              page1 = page_id(j + 2 + after);
            }
#pragma unroll
            for (int e = 0; e < NX; ++e)
              if (mine(e)) {
                const int i = cw + W_CONV * e + 32 * u, side = i >= PER_SIDE;
                const int row0 = (i & (PER_SIDE - 1)) * ROWS;
                const uint32_t f = __shfl_sync(0xffffffffu, side ? vf : kf, row0 >> c.ps_log2);
                uint4 w = cur[e];
                if ((left < W_KEYS && row0 + lrow >= left) || (bads >> (row0 >> c.ps_log2) & 1u)) w = make_uint4(0, 0, 0, 0);
                uint32_t x[8];
                codes16_half<FMT>(w, f, x);
                const uint32_t to = smem_u32(smem + S::KV_OFF + (2 * s + side) * S::TILE) + (row0 >> 3) * 1024 + lane_to;
                sts128(to, x[0], x[1], x[2], x[3]);
                sts128(to ^ 16, x[4], x[5], x[6], x[7]);
              }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[s]);
        }
      }
      if (!ok && lane == 0) set_device_err(DERR_WAIT_TIMEOUT);
  } else {
    // -------------------------------------------------- softmax of a tile
    const int a = (warp >> 2) - 1, qw = warp & 3, r = qw * 32 + lane;
    const uint32_t tl = tmem + a * 256 + ((uint32_t)(qw * 32) << 16);
    const float sl2 = LOG2E_F * (D == 64 ? 0.125f : 0.08838834764831845f);
    uint32_t g = 0, t = 0;
    bool ok = true;
    while (ok && at < end) {
      const Item p = item_at(k, pre, at, end);
      at = p.next;
      const int rows = p.q * k.group - p.row0 - a * 128;  // of this tile and those after it
      if (rows <= 0) {
        g += p.b1 - p.b0;
        continue;
      }
      if (p.b1 == p.b0) continue;
      const bool on = r < rows;
      const int row = p.row0 + a * 128 + (on ? r : 0), tok = row / k.group, h = p.head * k.group + row - tok * k.group;
      // the last token that the row sees, and the tile's first row, which sees the fewest, from this part's first block on
      int last = p.len - p.q + tok - p.b0 * W_KEYS;
      int first_last = p.len - p.q + (p.row0 + a * 128) / k.group - p.b0 * W_KEYS;
      const bool whole = p.b0 == 0 && p.b1 == p.blocks, begins = p.b0 == 0;
      const int out_row = p.a + tok;
      // ---- Q: the row times a power of two, as f16
      float rowf;
      {
        const uint4* src = reinterpret_cast<const uint4*>(k.q + (long)(p.a + tok) * k.ldq + h * D);
        uint4 x[D / 8];
        uint32_t mx = 0;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          x[e] = on ? src[e] : make_uint4(0, 0, 0, 0);
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[e].x & 0x7fff7fffu, x[e].y & 0x7fff7fffu),
                                     __vmaxu2(x[e].z & 0x7fff7fffu, x[e].w & 0x7fff7fffu)));
        }
        const int E = max((int)(max(mx & 0xffffu, mx >> 16) >> 7), 15);
        const float up = __uint_as_float((uint32_t)(268 - E) << 23);
        rowf = __uint_as_float((uint32_t)(E - 14) << 23) * sl2;
        const uint32_t dst = smem_u32(smem + a * S::TILE);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_bf16x2(w[i]);
            y[i] = half2_of(f.x * up, f.y * up);
          }
          sts128(dst + (e >> 3) * 16384 + sw128(r, e & 7), y[0], y[1], y[2], y[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[a]);
      }
      // the key scale from which on a score of the warp's rows may pass 2^20 (as bits: a block apart has the sign's)
      const uint32_t far_from = __float_as_uint(0x1p-10f / __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rowf))));
      float m = -INFINITY, l = 0.f, vref = 0.f;
      const int blocks = p.b1 - p.b0;
      for (int j = 0; ok && j < blocks;) {
        bool far = false;
        for (; j < blocks; ++j, ++g, ++t, last -= W_KEYS, first_last -= W_KEYS) {
          if (!warp_wait(&s_full[a], t & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const volatile float2* at_info = &info[g % NS];
          const float2 scale = make_float2(at_info->x, at_info->y);
          const float fs = fmaxf(scale.x * rowf, 1e-37f);  // (not 0: a masked score stays -inf)
          const bool edge = first_last < W_KEYS - 1;
          // The scores are read in quarters of 32; the last two twice, for the
          // maximum and for the weights.  With all 128 kept in registers the
          // other warps would have too few (spilled, each load would wait).
          float mx8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mx8[i] = -INFINITY;
          uint32_t x[3][32];
          auto masked = [&](uint32_t (&v)[32], int q) {
            if (edge) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * q + e > last) v[e] = __float_as_uint(-INFINITY);
            }
          };
          auto maximum = [&](uint32_t (&v)[32]) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float& y = mx8[(e >> 1) & 7];
              y = fmax3(y, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            }
          };
          tmem_ld32(tl + 64, x[0]);
          tmem_ld32(tl + 96, x[1]);
          tmem_wait_ld();
          far = __float_as_uint(scale.x) > far_from;
          if (far) break;
          masked(x[0], 2);
          maximum(x[0]);
          tmem_ld32(tl, x[0]);
          masked(x[1], 3);
          maximum(x[1]);
          tmem_ld32(tl + 32, x[1]);
          tmem_wait_ld();
          tmem_ld32(tl + 64, x[2]);
          masked(x[0], 0);
          maximum(x[0]);
          masked(x[1], 1);
          maximum(x[1]);
          const float mx = fs * fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                      fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
          // the reference moves when a row passes it by 2^8, and O also when the value scale rises
          const bool moved = __any_sync(0xffffffffu, mx > m + 8.f);
          const bool rescale = moved || scale.y > vref;
          float alpha = 1.f;
          if (moved) {
            const float nm = fmaxf(m, mx);
            alpha = m == -INFINITY ? 0.f : ex2f(m - nm);
            m = nm;
            l *= alpha;
          }
          if (scale.y > vref) {
            alpha *= vref / scale.y;
            vref = scale.y;
          }
          const float off = m == -INFINITY ? 0.f : m - 6.f;  // weights up to 2^14 in f16, down to 2^-30 of the reference
          // P's place is free, and O complete, once the block before has been multiplied
          if (j > 0 && !warp_wait(&pv_done[a], (t - 1) & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 fs2 = make_float2(fs, fs), off2 = make_float2(-off, -off);
          auto weights = [&](uint32_t (&v)[32], int q) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int e = 16 * half + 2 * i;
                float2 z = fma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), fs2, off2);
                z = make_float2(ex2f(z.x), ex2f(z.y));
                sum[i & 1] = add2(sum[i & 1], z);
                y[i] = half2_of(z.x, z.y);
              }
              tmem_st8(tl + S::T_P + 16 * q + 8 * half, y);
            }
          };
          weights(x[0], 0);
          tmem_ld32(tl + 96, x[0]);
          weights(x[1], 1);
          tmem_wait_ld();
          if (D == 64) {  // S is read: the next block's scores may be formed meanwhile
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[a]);
          }
          masked(x[2], 2);
          weights(x[2], 2);
          masked(x[0], 3);
          weights(x[0], 3);
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          if (j > 0 && rescale) {
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(tl + S::T_O + q * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tl + S::T_O + q * 32, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[a]);
        }
        if (!far) break;
        const volatile float2* at_info = &info[g % NS];
        FarRow row{m, l, vref, rowf};
        const float2 scale = make_float2(at_info->x, at_info->y);
        ok = far_block<D>(row, tl, scale, &apart_at[(g % NS) * 8], c.ps_log2, last, j > 0 ? &pv_done[a] : nullptr, (t - 1) & 1u);
        if (ok && lane == 0) {
          if (D == 64) mbar_arrive(&s_free[a]);
          mbar_arrive(&p_full[a]);
        }
        m = row.m, l = row.l, vref = scale.y;
        // the rows' O to one reference again, in fp32
        if (ok && __any_sync(0xffffffffu, row.vref != vref)) {
          ok = warp_wait(&pv_done[a], t & 1u);
          if (ok) far_rescale<D>(tl, row.vref / vref);
        }
        ++j, ++g, ++t, last -= W_KEYS, first_last -= W_KEYS;
      }
      if (!ok || !warp_wait(&pv_done[a], (t - 1) & 1u)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // ---- the item's result, or this part's share of it
      float* part = k.part + ((long)blockIdx.x * 2 + begins) * W_ROWS * (D + 2);
      const int pr = a * 128 + r;
      const float M = m - 6.f;  // the sums' reference
      const float f = whole ? vref / l : vref;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(tl + S::T_O + q * 32, o);
        tmem_wait_ld();
        if (on && whole) {
          uint4* dst = reinterpret_cast<uint4*>(k.out + (long)out_row * k.ldo + h * D + q * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * i]) * f, __uint_as_float(o[8 * i + 1]) * f),
                                pack_bf16x2(__uint_as_float(o[8 * i + 2]) * f, __uint_as_float(o[8 * i + 3]) * f),
                                pack_bf16x2(__uint_as_float(o[8 * i + 4]) * f, __uint_as_float(o[8 * i + 5]) * f),
                                pack_bf16x2(__uint_as_float(o[8 * i + 6]) * f, __uint_as_float(o[8 * i + 7]) * f));
        } else if (on) {
          float4* dst = reinterpret_cast<float4*>(part + pr * D + q * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(o[4 * i]) * f, __uint_as_float(o[4 * i + 1]) * f,
                                 __uint_as_float(o[4 * i + 2]) * f, __uint_as_float(o[4 * i + 3]) * f);
        }
      }
      tc_fence_before();
      if (on && !whole) {
        part[W_ROWS * D + pr] = M;
        part[W_ROWS * D + W_ROWS + pr] = l;
      }
      if (on && whole && k.lse) k.lse[(long)out_row * k.H + h] = (M + log2f(l)) * 0.6931471805599453f;
    }
    if (!ok) set_device_err(DERR_WAIT_TIMEOUT);
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// The rows behind `row0` of the item that begins in part x and goes on after
// it, four columns of a row per thread; four parts are requested at once.
constexpr int J_THREADS = 32 * J_WARPS;
template <int D>
__device__ __forceinline__ void join_item(const Call& k, int part_x, int row0) {
  const Join t = k.join[part_x];
  const int r = row0 + threadIdx.x / (D / 4), d4 = threadIdx.x % (D / 4);
  if (r >= t.tile_rows || t.parts == 0) return;
  constexpr long SIZE = (long)W_ROWS * (D + 2);
  const float* first = k.part + ((long)part_x * 2 + 1) * SIZE;
  float M = -INFINITY, L = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < t.parts; j0 += 4) {
    float m[4], l[4];
    float4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u;
      const float* src = first + (j ? (2 * j - 1) * SIZE : 0);
      m[u] = -INFINITY, l[u] = 0.f, x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < t.parts) {
        m[u] = src[W_ROWS * D + r];
        l[u] = src[W_ROWS * D + W_ROWS + r];
        x[u] = *reinterpret_cast<const float4*>(src + r * D + 4 * d4);
      }
    }
    const float nm = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), M);
    const float nu = nm == -INFINITY ? 0.f : nm;
    const float f = ex2_approx(M - nu);
    M = nm;
    L *= f, a.x *= f, a.y *= f, a.z *= f, a.w *= f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float h = ex2_approx(m[u] - nu);
      L += h * l[u];
      a.x += h * x[u].x, a.y += h * x[u].y, a.z += h * x[u].z, a.w += h * x[u].w;
    }
  }
  const float inv = 1.f / L;
  const int row = t.row0 + r, tok = row / k.group, h = t.head * k.group + row - tok * k.group;
  *reinterpret_cast<uint2*>(k.out + (long)(t.a + tok) * k.ldo + h * D + 4 * d4) =
      make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (d4 == 0 && k.lse) k.lse[(long)(t.a + tok) * k.H + h] = (M + log2f(L)) * 0.6931471805599453f;
}

// Joins the items of the wide kernel and the tiles of the streaming kernel that
// followed it, in one launch: first `parts` CTAs for every J_THREADS threads of
// an item, then CTAs that list the cut tiles among `narrow_parts` and take the
// join_ctas shares of each in turn (a CTA per share of every part would be 2368
// CTAs, nearly all of them empty).
template <int D>
__global__ void __launch_bounds__(J_THREADS) join_wide_kernel(const Call k, const Join* narrow, const float* narrow_part,
                                                              int parts, int narrow_parts) {
  constexpr int ROWS = J_THREADS / (D / 4), CTAS = W_ROWS / ROWS;
  static_assert(CTAS * ROWS == W_ROWS, "every row of an item has its threads");
  pdl_wait();
  const int b = blockIdx.x;
  if (b < parts * CTAS) {
    join_item<D>(k, b % parts, b / parts * ROWS);
    return;
  }
  extern __shared__ int s_cut[];  // [narrow_parts]
  __shared__ int s_count[J_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int count = 0;
  for (int i0 = 0; i0 < narrow_parts; i0 += J_THREADS) {
    const int i = i0 + threadIdx.x;
    const bool cut = i < narrow_parts && narrow[i].parts > 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, cut);
    if (lane == 0) s_count[warp] = __popc(mask);
    __syncthreads();
    int at = count + __popc(mask & ((1u << lane) - 1));
    for (int w = 0; w < J_WARPS; ++w) {
      if (w < warp) at += s_count[w];
      count += s_count[w];
    }
    if (cut) s_cut[at] = i;
    __syncthreads();
  }
  constexpr int RT = wide_row_tile(D);
  for (int u = b - parts * CTAS; u < count * join_ctas(RT); u += gridDim.x - parts * CTAS)
    join_tile<D, RT>(k, narrow, narrow_part, s_cut[u / join_ctas(RT)], u % join_ctas(RT));
}

static inline size_t wide_workspace_bytes(const Cache& c) {
  return (size_t)sm_count() * (sizeof(Join) + 2 * (size_t)W_ROWS * (c.d + 2) * 4);
}

// The streaming kernel for the call's short sequences starts on the SMs that
// the wide kernel leaves; each kernel of the chain ends after the one before it.
// One join for both: 2 us less than one for each.
template <int FMT, int D>
static inline cudaError_t wide_launch(const Call& k, void* work, void* stream_work, cudaStream_t st) {
  using S = Wide<D>;
  static DeviceOnce once;
  cudaError_t e = run_once_per_device(once, [] {
    return cudaFuncSetAttribute(wide_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::bytes(MAX_SEQS));
  });
  if (e != cudaSuccess) return e;
  const int grid = sm_count();
  Call a = k;
  a.join = static_cast<Join*>(work);
  a.part = reinterpret_cast<float*>(a.join + grid);
  a.setup = 12;     // an item's Q, first scores and output: three blocks' time
  a.min_part = 20;
  wide_kernel<FMT, D><<<grid, W_THREADS, S::bytes(k.n), st>>>(a);
  e = cudaGetLastError();
  if (e == cudaSuccess && k.narrow) e = stream(k, stream_work, st, true);
  if (e != cudaSuccess) return e;
  constexpr int RT = wide_row_tile(D), CTAS = W_ROWS * (D / 4) / J_THREADS;
  const int parts = k.narrow && !whole_tiles(k.c) ? parts_of(k.c, RT) : 0;
  const Join* join = static_cast<const Join*>(stream_work);
  return launch_after(join_wide_kernel<D>, dim3(grid * CTAS + parts), J_THREADS, parts * sizeof(int), st, a, join,
                      reinterpret_cast<const float*>(join + parts), grid, parts);
}

static inline cudaError_t wide(const Call& k, void* work, void* stream_work, cudaStream_t st) {
  if (k.c.fmt == GPT2_KV_INT8)
    return k.c.d == 64 ? wide_launch<GPT2_KV_INT8, 64>(k, work, stream_work, st)
                       : wide_launch<GPT2_KV_INT8, 128>(k, work, stream_work, st);
  return k.c.d == 64 ? wide_launch<GPT2_KV_E4M3, 64>(k, work, stream_work, st)
                     : wide_launch<GPT2_KV_E4M3, 128>(k, work, stream_work, st);
}

// ---------------------------------------------------------------- the call
// One sequence: whichever kernel suits max_q takes it, whatever its rows.
// More: each sequence goes by its own rows, so that single tokens and prompts
// may share a call; without a prompt (max_q) the wide kernel is not launched.
static inline int narrow_limit(int group, int n, int max_q) {
  return (long)group * max_q <= NARROW_ROWS ? NARROW_ROWS : n == 1 ? 0 : NARROW_ROWS;
}

static inline size_t attention_workspace_bytes(const Cache& c, int H, int n, int, int max_q) {
  const int group = H / c.kvh;
  return (narrow_limit(group, n, max_q) ? stream_workspace_bytes(c, H, max_q) : 0) +
         ((long)group * max_q > NARROW_ROWS ? wide_workspace_bytes(c) : 0);
}

static inline cudaError_t attention(const Cache& c, int layer, const bf16* q, long ldq, bf16* out, long ldo,
                                    float* lse, int H, const int32_t* slots, const int32_t* cu, int n, int rows,
                                    int max_q, void* work, cudaStream_t st) {
  Call k;
  k.c = c;
  k.layer = layer;
  k.H = H;
  k.group = H / c.kvh;
  k.n = n;
  k.rows = rows;
  k.max_q = max_q < rows ? max_q : rows;
  k.q = q;
  k.ldq = ldq;
  k.out = out;
  k.ldo = ldo;
  k.lse = lse;
  k.slots = slots;
  k.cu = cu;
  k.join = nullptr;
  k.part = nullptr;
  k.narrow = narrow_limit(k.group, n, max_q);
  k.setup = k.min_part = 0;
  k.zero = 0;
  if ((long)k.group * max_q <= NARROW_ROWS) return stream(k, work, st, false);
  return wide(k, work, static_cast<uint8_t*>(work) + wide_workspace_bytes(c), st);
}

}  // namespace kv8

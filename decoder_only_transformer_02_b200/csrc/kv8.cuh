// Paged key/value cache held in 8 bits: the layout, the page table's
// operations (resize, fork, compact) and the append that rounds new keys and
// values into it.  The attention that reads it is in kv8_attention.cuh.
//
// A page holds page_size tokens of every layer:
//   codes  [num_pages][n_layer][2][n_kv_head][page_size][head_dim]  8 bits (side 0 keys, 1 values)
//   scales [num_pages][n_layer][2][n_kv_head]                       fp32, powers of two
// so a page is one contiguous block (copied by fork and compact as such) and
// the tokens of one (page, layer, side, head) are one contiguous tile, which
// the attention streams.  A value is code * scale.
//   table  [num_slots][max_pages]  page ids of a slot's tokens, in order
//   lens   [num_slots]             cached tokens of a slot
//   refs   [num_pages]             slots that hold the page (0: free)
//
// Why powers of two: x / scale is then exact, so a code is one rounding of the
// value itself, and the codes do not depend on how the division was computed;
// when a page's scale grows, e4m3 codes move by whole exponents (exact down to
// their subnormals).  The price is up to one bit of the int8 range (scale up
// to 2 * amax / 127).  The smallest scale is 2^-126.
#pragma once
#include "../../include/gpt2.h"
#include "common.cuh"

namespace kv8 {

constexpr int MAX_SEQS = 4096;      // entries of one call (their offsets are scanned in shared memory)
constexpr int MAX_SLOTS = 1 << 16;  // the duplicate check's bitmap is 8 KB of shared memory
constexpr int MAX_PAGES = 1 << 24;
constexpr int MAX_TOKENS = 1 << 30;  // of a slot
constexpr int MAX_ROWS = 1 << 24;    // of a call
constexpr uint32_t NAN_SCALE = 0x7fc00000u;

struct Cache {
  int fmt, L, kvh, d, ps, ps_log2, num_pages, num_slots, max_pages;
  uint8_t* codes;
  float* scales;
  int32_t *table, *lens, *refs;
  __host__ __device__ long tile() const { return (long)ps * d; }                     // bytes of one head's tokens
  __host__ __device__ long page_bytes() const { return 2L * L * kvh * ps * d; }
  __host__ __device__ int page_scales() const { return 2 * L * kvh; }
  // index of (page, layer, side, head) among the tiles and scales
  __device__ __forceinline__ long unit(int page, int layer, int side, int head) const {
    return (((long)page * L + layer) * 2 + side) * kvh + head;
  }
  __device__ __forceinline__ bool page_ok(int p) const { return (unsigned)p < (unsigned)num_pages; }
  __device__ __forceinline__ int pages_of(int len) const { return (int)(((long)len + ps - 1) >> ps_log2); }
  // length of a slot; -1 (flagged) when the slot or its length is out of range
  __device__ __forceinline__ int len_of(int slot) const {
    if ((unsigned)slot >= (unsigned)num_slots) return -1;
    const int len = lens[slot];
    return len < 0 || pages_of(len) > max_pages ? -1 : len;
  }
};

// The caller's description as the kernels take it; false where a size or
// pointer is out of its limits.
static inline bool cache_of(const gpt2_kv8* k, Cache& c) {
  if (!k || !k->d_codes || !k->d_scales || !k->d_table || !k->d_lens || !k->d_refs) return false;
  if (k->format != GPT2_KV_INT8 && k->format != GPT2_KV_E4M3) return false;
  if (k->n_layer < 1 || k->n_layer > 1024 || k->n_kv_head < 1 || k->n_kv_head > 1024) return false;
  if (k->head_dim != 64 && k->head_dim != 128) return false;
  if (k->page_size != 16 && k->page_size != 32 && k->page_size != 64 && k->page_size != 128) return false;
  if (k->num_pages < 1 || k->num_pages > MAX_PAGES || k->num_slots < 1 || k->num_slots > MAX_SLOTS) return false;
  if (k->max_pages < 1 || (long)k->max_pages * k->page_size > MAX_TOKENS) return false;
  if ((reinterpret_cast<uintptr_t>(k->d_codes) & 15) || (reinterpret_cast<uintptr_t>(k->d_refs) & 15)) return false;
  c.fmt = k->format;
  c.L = k->n_layer;
  c.kvh = k->n_kv_head;
  c.d = k->head_dim;
  c.ps = k->page_size;
  c.ps_log2 = k->page_size == 16 ? 4 : k->page_size == 32 ? 5 : k->page_size == 64 ? 6 : 7;
  c.num_pages = k->num_pages;
  c.num_slots = k->num_slots;
  c.max_pages = k->max_pages;
  c.codes = (uint8_t*)k->d_codes;
  c.scales = k->d_scales;
  c.table = k->d_table;
  c.lens = k->d_lens;
  c.refs = k->d_refs;
  return true;
}

// griddepcontrol: the second kernel of a pair is launched while the first
// runs and waits here for its results
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------------- append
// Rounding of the new tokens of one (page, layer, side, head), by one warp:
//   amax over the new values; scale' = 2^e, the smallest (e >= -126) with
//   amax <= qmax 2^e, or the page's old scale if that is larger and the page
//   already holds older tokens; codes round(x / scale') to nearest even.
// A scale that grows rescales the whole tile's codes first.  A value that is
// not finite makes the scale NaN: the block then reads as NaN.
__device__ __forceinline__ uint32_t scale_bits_for(uint32_t amax_bf16, int fmt) {
  const int E = (int)(amax_bf16 >> 7), m = (int)(amax_bf16 & 127);
  if (E == 255) return NAN_SCALE;
  // 127 = (1 + 126/128) 2^6, 448 = (1 + 96/128) 2^8; the exponent field of scale'
  const int e = fmt == GPT2_KV_INT8 ? E - (m <= 126 ? 6 : 5) : E - (m <= 96 ? 8 : 7);
  return (uint32_t)max(e, 1) << 23;
}
// 1 / scale of a power of two from 2^-126 to 2^126 (exponent fields 1..253)
__device__ __forceinline__ float inverse_pow2(uint32_t bits) { return __uint_as_float(0x7f000000u - bits); }

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
template <int FMT>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  if (FMT == GPT2_KV_E4M3) return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
  // adding 1.5 * 2^23 rounds to the nearest integer (even on ties), in the low bits
  const uint32_t x = __float_as_uint(a + 12582912.f), y = __float_as_uint(b + 12582912.f);
  const uint32_t z = __float_as_uint(c + 12582912.f), w = __float_as_uint(d + 12582912.f);
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}
template <int FMT>
__device__ __forceinline__ void unpack4(uint32_t w, float (&f)[4]) {
  if (FMT == GPT2_KV_E4M3) {
    const uint32_t lo = e4m3x2_to_half2(w & 0xffffu), hi = e4m3x2_to_half2(w >> 16);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
  }
}

constexpr int APPEND_WARPS = 8;

// CTA (x, y): x names a run of one sequence's new tokens inside one page, whose
// 2 * kvh (side, head) pairs the warps of the CTAs (x, *) share.
// by_row: x is a row, and works if its token is the run's first.  Otherwise x
// counts runs: sequence i owns the numbers from cu[i] / ps + 2 i, enough since
// its q tokens touch at most q / ps + 2 pages; no prefix sum is needed.
// HELD: 16-byte pieces of a tile that a lane keeps between the two passes: 1 for
// short runs, 4 (a tile of 1024 values) for prompts; the rest is read again, UN
// pieces at a time: 1 where nothing is left (17.9 us; with 4, whose registers
// cost warps, 20.0), 4 where tiles are larger (64 tokens of 64: 22.5; with 1, 30).
// What it moves: 2 bytes in, 1 out per value.  15,400 rows of 2 x 768 values:
// 17.9 us (3.9 TB/s; 25.7 with both passes reading, 22 with 8 pieces held, whose
// registers cost half the warps); 256 single rows: 5.8 us, its chain of loads.
template <int FMT, int HELD, int UN>
__global__ void __launch_bounds__(32 * APPEND_WARPS)
    append_kernel(Cache c, int layer, const bf16* __restrict__ k, const bf16* __restrict__ v, long ld,
                  const int32_t* __restrict__ slots, const int32_t* __restrict__ cu, int n, int rows, int by_row) {
  __shared__ int s_i, s_a, s_b, s_slot;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int x = blockIdx.x;
  if (tid == 0) s_i = -1;
  __syncthreads();
  bool bad = false;
#pragma unroll 1
  for (int i = tid; i < n; i += blockDim.x) {
    const int a = cu[i], b = cu[i + 1], slot = slots[i];
    const bool mine = by_row ? x >= a && x < b
                             : x >= (a >> c.ps_log2) + 2 * i && x < (b >> c.ps_log2) + 2 * i + 2;
    bad |= a < 0 || b < a || b > rows;
    if (mine) s_i = i, s_a = a, s_b = b, s_slot = slot;  // one thread at most, unless the offsets are bad
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_device_err(DERR_KV8_ARGS);
    return;
  }
  const int i = s_i;
  if (i < 0) return;
  const int a = s_a, q = s_b - a, slot = s_slot;
  const int len = c.len_of(slot);
  // a slot named twice: the later entries are refused, or both would write the same tokens
  bool twice = false;
#pragma unroll 1
  for (int j = tid; j < i; j += blockDim.x) twice |= slots[j] == slot && cu[j + 1] > cu[j];
  twice = __syncthreads_or(twice);
  if (q == 0) return;
  if (len < q || twice) {
    if (tid == 0) set_device_err(DERR_KV8_ARGS);
    return;
  }
  const int p0 = len - q;  // position of the sequence's first new token
  int pos, end;
  if (by_row) {
    pos = p0 + (x - a);
    if (x != a && (pos & (c.ps - 1)) != 0) return;
  } else {
    const int j = x - ((a >> c.ps_log2) + 2 * i);
    pos = j == 0 ? p0 : ((p0 >> c.ps_log2) + j) << c.ps_log2;
    if (pos >= len) return;
  }
  end = min(len, (pos | (c.ps - 1)) + 1);
  const int page = c.table[(long)slot * c.max_pages + (pos >> c.ps_log2)];
  if (!c.page_ok(page)) {
    if (tid == 0) set_device_err(DERR_KV8_TABLE);
    return;
  }
  // (looked at behind the rows' loads, which it would otherwise keep waiting)
  const int holders = __ldcg(c.refs + page);
  const int d8 = c.d >> 3, m = end - pos;       // 16-byte pieces of a row; rows
  const int per = 32 / d8, sub = lane / d8;     // rows a warp reads at once; this lane's
  const int off = pos & (c.ps - 1);
#pragma unroll 1
  for (int pair = blockIdx.y * APPEND_WARPS + warp; pair < 2 * c.kvh; pair += gridDim.y * APPEND_WARPS) {
    const int side = pair >= c.kvh, head = pair - side * c.kvh;
    const long u = c.unit(page, layer, side, head);
    const bf16* src = (side ? v : k) + (long)(a + pos - p0) * ld + head * c.d + (lane % d8) * 8;
    uint8_t* tile = c.codes + u * c.tile();
    // the largest magnitude, as bf16 bits (their order is the values')
    uint4 x[HELD];
    uint32_t mx = 0;
    auto largest = [&](const uint4& w) {
      const uint32_t t0 = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
      const uint32_t t1 = __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu);
      mx = __vmaxu2(mx, __vmaxu2(t0, t1));
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (sub + i * per < m) x[i] = __ldg(reinterpret_cast<const uint4*>(src + (long)(sub + i * per) * ld));
    }
    const uint32_t old = off ? __float_as_uint(c.scales[u]) : 0u;
#pragma unroll UN
    for (int r = sub + HELD * per; r < m; r += per) largest(__ldg(reinterpret_cast<const uint4*>(src + (long)r * ld)));
#pragma unroll
    for (int i = 0; i < HELD; ++i) largest(x[i]);
    mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    if (holders != 1) {  // a page that other slots read too, or that is free
      if (lane == 0) set_device_err(DERR_KV8_TABLE);
      return;
    }
    uint32_t bits = scale_bits_for(mx, FMT);
    if (off != 0) {
      if (bits > old && bits != NAN_SCALE) {  // positive floats and the NaN order as their bits
        const float ratio = __uint_as_float(old) * inverse_pow2(bits);
#pragma unroll 1
        for (int t = lane; t < (int)(c.tile() >> 4); t += 32) {
          uint4 w = reinterpret_cast<uint4*>(tile)[t];
          uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float f[4];
            unpack4<FMT>(e[g], f);
            e[g] = pack4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
          }
          reinterpret_cast<uint4*>(tile)[t] = make_uint4(e[0], e[1], e[2], e[3]);
        }
      }
      bits = max(bits, old);
    }
    __syncwarp();  // every lane has read the old scale, and the rescaled codes come before the new ones
    if (lane == 0) c.scales[u] = __uint_as_float(bits);
    const bool nan = bits >= NAN_SCALE;
    const float inv = nan ? 0.f : inverse_pow2(bits);
    uint8_t* dst = tile + (long)off * c.d + (lane % d8) * 8;
    auto store = [&](const uint4& w, int r) {
      const float2 f0 = unpack_bf16x2(w.x), f1 = unpack_bf16x2(w.y), f2 = unpack_bf16x2(w.z), f3 = unpack_bf16x2(w.w);
      uint2 o;
      o.x = pack4<FMT>(f0.x * inv, f0.y * inv, f1.x * inv, f1.y * inv);
      o.y = pack4<FMT>(f2.x * inv, f2.y * inv, f3.x * inv, f3.y * inv);
      if (nan) o = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(dst + r * c.d) = o;
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (sub + i * per < m) store(x[i], sub + i * per);
#pragma unroll UN
    for (int r = sub + HELD * per; r < m; r += per) store(__ldg(reinterpret_cast<const uint4*>(src + (long)r * ld)), r);
    __syncwarp();
  }
}

constexpr long APPEND_CTAS = 148 * 4;
static inline cudaError_t append(const Cache& c, int layer, const bf16* k, const bf16* v, long ld,
                                 const int32_t* slots, const int32_t* cu, int n, int rows, cudaStream_t st) {
  if (n == 0 || rows == 0) return cudaSuccess;
  const long runs = (long)(rows >> c.ps_log2) + 2L * n;
  const int by_row = rows <= runs;
  const long xs = by_row ? rows : runs;
  // finding its run costs a CTA four dependent loads: with runs enough for
  // APPEND_CTAS, more of the pairs go to one CTA
  const int most = (2 * c.kvh + APPEND_WARPS - 1) / APPEND_WARPS;
  const int ys = (int)(xs * most <= APPEND_CTAS ? most : (APPEND_CTAS + xs - 1) / xs);
  const dim3 grid((unsigned)xs, ys < 1 ? 1 : ys > most ? most : ys);
#define KV8_APPEND(F, HELD, UN) \
  append_kernel<F, HELD, UN><<<grid, 32 * APPEND_WARPS, 0, st>>>(c, layer, k, v, ld, slots, cu, n, rows, by_row)
  const bool fits = c.tile() <= 1024;
  if (c.fmt == GPT2_KV_INT8)
    by_row ? KV8_APPEND(GPT2_KV_INT8, 1, 1) : fits ? KV8_APPEND(GPT2_KV_INT8, 4, 1) : KV8_APPEND(GPT2_KV_INT8, 4, 4);
  else
    by_row ? KV8_APPEND(GPT2_KV_E4M3, 1, 1) : fits ? KV8_APPEND(GPT2_KV_E4M3, 4, 1) : KV8_APPEND(GPT2_KV_E4M3, 4, 4);
#undef KV8_APPEND
  return cudaGetLastError();
}

// ------------------------------------------------- page table: plan and apply
// resize, fork and compact run as two kernels.  The plan (one CTA) checks the
// arguments, so that a refused call changes nothing, and finds the pages: free
// pages are handed out lowest first, in the order of the list.  The apply
// kernel (many CTAs) rewrites the tables and counts and copies the pages.
// One CTA plans because the hand-out is a prefix sum over the pool: 3 to 5 us for
// pools of some thousand pages, most of it dependent loads, 0.7 us more for each
// further 4096 pages that it has to look through.
// The workspace (32-bit words):
//   head[16]: 0 go, 1 copies, 2 pages wanted, 3 live pages, 4 live pages below the live count
//   first[n]: the number of pages wanted by the entries before
//   copy[2 n]: source page and destination's number among the free pages of each copy
//   list[3 num_pages]: free pages in order; (compact) holes, high pages by live rank, live rank of a page
constexpr int HEAD = 16;
constexpr int PLAN_THREADS = 1024;

struct Work {
  int32_t *head, *first, *copy, *list, *high, *rank;
};
static inline Work work_of(void* w, int n, int num_pages) {
  int32_t* p = static_cast<int32_t*>(w);
  Work k;
  k.head = p;
  k.first = p + HEAD;
  k.copy = k.first + n;
  k.list = k.copy + 2L * n;
  k.high = k.list + num_pages;
  k.rank = k.high + num_pages;
  return k;
}
// where a resize or fork with this workspace leaves whether it went through (0: refused)
static inline const int32_t* go_word(const void* w) { return static_cast<const int32_t*>(w); }
static inline size_t workspace_bytes(int n, int num_pages) { return 4 * (HEAD + 3 * (size_t)n + 3 * (size_t)num_pages); }

// exclusive prefix sum over the block; `total` receives the sum
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t& total, uint64_t* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // s_warp is free again
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  uint64_t w = s_warp[lane];  // every warp adds up the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const uint64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return x - v + (warp ? before : 0);
}

// four page counts from p on (1 behind the pool's end)
__device__ __forceinline__ int4 refs_at(const Cache& c, int p) {
  int4 r = make_int4(1, 1, 1, 1);
  if (p + 3 < c.num_pages) return __ldcg(reinterpret_cast<const int4*>(c.refs + p));
  if (p < c.num_pages) r.x = __ldcg(c.refs + p);
  if (p + 1 < c.num_pages) r.y = __ldcg(c.refs + p + 1);
  if (p + 2 < c.num_pages) r.z = __ldcg(c.refs + p + 2);
  return r;
}

// A pass over the pool takes 4 x 4096 pages at a time: thread t the pages 4 t ..
// + 3 of each 4096, and one scan of the four counts, 16 bits each.
constexpr int SCAN = 4 * PLAN_THREADS;
struct Four {
  int4 r[4];
};
__device__ __forceinline__ Four four_at(const Cache& c, int base) {
  Four f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f.r[q] = make_int4(1, 1, 1, 1);
    if (base + q * SCAN < c.num_pages) f.r[q] = refs_at(c, base + q * SCAN + 4 * (int)threadIdx.x);
  }
  return f;
}

// The wanted lowest free pages (refs 0) into list; returns how many there are
// (at least `want`, or all of them).
__device__ __forceinline__ uint64_t find_free(const Cache& c, uint64_t want, int32_t* list, uint64_t* s_warp) {
  uint64_t found = 0;
  if (want == 0) return 0;
  Four f = four_at(c, 0);
  for (long base = 0; base < c.num_pages && found < want; base += 4 * SCAN) {
    uint64_t count = 0, total;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (base + q * SCAN < c.num_pages)
        count += (uint64_t)((f.r[q].x == 0) + (f.r[q].y == 0) + (f.r[q].z == 0) + (f.r[q].w == 0)) << (16 * q);
    const uint64_t before = block_scan(count, total, s_warp);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (base + q * SCAN >= c.num_pages) break;
      uint64_t at = found + (before >> (16 * q) & 0xffff);
      const int p = (int)base + q * SCAN + 4 * (int)threadIdx.x;
      const int v[4] = {f.r[q].x, f.r[q].y, f.r[q].z, f.r[q].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (v[e] == 0 && at < want) list[at] = p + e;
        at += v[e] == 0;
      }
      found += total >> (16 * q) & 0xffff;
    }
    if (base + 4 * SCAN < c.num_pages) f = four_at(c, (int)base + 4 * SCAN);
  }
  return found;
}

// What a resize does to one slot.
struct Change {
  int have, want, edge, copy, src;  // pages before and after; the page kept in part: its column, whether copied, its id
};
__device__ __forceinline__ Change change_of(const Cache& c, int slot, int old_len, int new_len) {
  Change h;
  h.have = c.pages_of(old_len);
  h.want = c.pages_of(new_len);
  const int keep = min(old_len, new_len);
  h.edge = keep >> c.ps_log2;
  h.copy = 0;
  h.src = -1;
  if (keep & (c.ps - 1)) {
    h.src = c.table[(long)slot * c.max_pages + h.edge];
    if (!c.page_ok(h.src))
      h.copy = -1;
    else
      h.copy = c.refs[h.src] > 1;
  }
  return h;
}

// Every slot in range and none named twice (a bitmap in shared memory).
__device__ __forceinline__ bool claim(const Cache& c, int slot, uint32_t* s_map) {
  if ((unsigned)slot >= (unsigned)c.num_slots) return false;
  return !(atomicOr(&s_map[slot >> 5], 1u << (slot & 31)) >> (slot & 31) & 1u);
}

// Shared memory of a plan: the slots' bitmap, and for a resize each entry's
// slot, pages kept and number of pages given back by the entries before.
static inline size_t plan_smem(const Cache& c, int n, bool resize) {
  return (size_t)((c.num_slots + 31) / 32 * 4 + 7) / 8 * 8 + (resize ? (size_t)n * 16 : 0);
}

__global__ void __launch_bounds__(PLAN_THREADS)
    resize_plan_kernel(Cache c, const int32_t* __restrict__ slots, const int32_t* __restrict__ lens, int n, Work w) {
  extern __shared__ __align__(16) uint32_t s_map[];
  __shared__ uint64_t s_warp[32];
  const int tid = threadIdx.x, words = (c.num_slots + 31) / 32;
  uint64_t* s_first = reinterpret_cast<uint64_t*>(s_map + (words + 1) / 2 * 2);  // [n]
  int2* s_entry = reinterpret_cast<int2*>(s_first + n);                          // [n]
  pdl_launch();
  for (int i = tid; i < words; i += PLAN_THREADS) s_map[i] = 0;
  __syncthreads();
  int err = 0;
  uint64_t want = 0, back = 0;  // pages wanted (and copies, from bit 40 on); pages given back
  for (int base = 0; base < n; base += PLAN_THREADS) {
    const int i = base + tid;
    uint64_t need = 0, drop = 0;
    int copy = 0, src = 0;
    if (i < n) {
      const int slot = slots[i], new_len = lens[i];
      const int old_len = c.len_of(slot);
      if (!claim(c, slot, s_map) || old_len < 0 || new_len < 0 || c.pages_of(new_len) > c.max_pages) {
        err = DERR_KV8_ARGS;
      } else {
        const Change h = change_of(c, slot, old_len, new_len);
        if (h.copy < 0) err = DERR_KV8_TABLE;
        copy = h.copy > 0, src = h.src;
        need = ((uint64_t)copy << 40) + copy + max(0, h.want - h.have);
        drop = max(0, h.have - h.want);
        s_entry[i] = make_int2(slot, h.want);
      }
    }
    uint64_t total;
    const uint64_t at = want + block_scan(need, total, s_warp);
    want += total;
    if (i < n) w.first[i] = (int)(at & 0x7fffffffu);  // (whole where the call goes on)
    if (copy) {
      w.copy[2 * (at >> 40)] = src;
      w.copy[2 * (at >> 40) + 1] = w.first[i];
    }
    const uint64_t before = back + block_scan(drop, total, s_warp);
    back += total;
    if (i < n) s_first[i] = before;
  }
  const uint64_t copies = want >> 40;
  want &= (1ull << 40) - 1;
  if (__syncthreads_or(err) != 0) {
    if (err) set_device_err(err);
    if (tid == 0) w.head[0] = 0;
    return;
  }
  for (int sign = -1; sign <= 1; sign += 2) {  // give back; a second time, with +1, only where too few are free
    for (uint64_t r = tid; r < back; r += PLAN_THREADS) {
      int lo = 0, hi = n;  // the entry of the r-th page given back
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_first[mid] <= r) lo = mid; else hi = mid;
      }
      const int2 e = s_entry[lo];
      const int page = c.table[(long)e.x * c.max_pages + e.y + (r - s_first[lo])];
      if (c.page_ok(page))
        atomicAdd(&c.refs[page], sign);
      else
        set_device_err(DERR_KV8_TABLE);
    }
    __syncthreads();
    if (sign > 0) {
      if (tid == 0) {
        set_device_err(DERR_KV8_PAGES);
        w.head[0] = 0;
      }
      return;
    }
    if (find_free(c, want, w.list, s_warp) >= want) break;
    __syncthreads();
  }
  if (tid == 0) {
    w.head[0] = 1;
    w.head[1] = (int)copies;
    w.head[2] = (int)want;
  }
}

__global__ void __launch_bounds__(PLAN_THREADS)
    fork_plan_kernel(Cache c, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n, Work w) {
  extern __shared__ __align__(16) uint32_t s_map[];
  __shared__ uint64_t s_warp[32];
  const int tid = threadIdx.x;
  pdl_launch();
  for (int i = tid; i < (c.num_slots + 31) / 32; i += PLAN_THREADS) s_map[i] = 0;
  __syncthreads();
  int err = 0;
  uint64_t want = 0;
  for (int base = 0; base < n; base += PLAN_THREADS) {
    const int i = base + tid;
    int part = 0, page = 0;
    if (i < n) {
      const int len = c.len_of(src[i]);
      if (len < 0 || !claim(c, dst[i], s_map) || c.lens[dst[i]] != 0) {
        err = DERR_KV8_ARGS;
      } else if (len & (c.ps - 1)) {
        part = 1;
        page = c.table[(long)src[i] * c.max_pages + (len >> c.ps_log2)];
        if (!c.page_ok(page)) err = DERR_KV8_TABLE;
      }
    }
    uint64_t total;
    const int at = (int)(want + block_scan(part, total, s_warp));
    if (i < n) w.first[i] = at;
    if (part) {
      w.copy[2 * at] = page;
      w.copy[2 * at + 1] = at;
    }
    want += total;
  }
  // a source that is also a destination would be read while it is written
  __syncthreads();
  for (int i = tid; i < n && err == 0; i += PLAN_THREADS)
    if (s_map[src[i] >> 5] >> (src[i] & 31) & 1u) err = DERR_KV8_ARGS;
  bool ok = __syncthreads_or(err) == 0;
  if (ok && find_free(c, want, w.list, s_warp) < want) {
    ok = false;
    if (tid == 0) err = DERR_KV8_PAGES;
  }
  if (err) set_device_err(err);
  if (tid == 0) {
    w.head[0] = ok;
    w.head[1] = (int)want;
    w.head[2] = (int)want;
  }
}

// n_live = pages with refs > 0.  The j-th live page with an id of n_live or
// more moves to the j-th free page below n_live.  high[live rank] is written
// for the pages that move, rank[id] for all from n_live on (-1: free), list[j]
// for the holes.
__global__ void __launch_bounds__(PLAN_THREADS) compact_plan_kernel(Cache c, Work w) {
  __shared__ uint64_t s_warp[32];
  const int tid = threadIdx.x;
  pdl_launch();
  auto used = [&](int p, int refs) { return p < c.num_pages && refs > 0; };
  Four f = four_at(c, 0);
  uint64_t count = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int p = q * SCAN + 4 * tid;
    count += used(p, f.r[q].x) + used(p + 1, f.r[q].y) + used(p + 2, f.r[q].z) + used(p + 3, f.r[q].w);
  }
#pragma unroll 4
  for (int p = 4 * SCAN + 4 * tid; p < c.num_pages; p += SCAN) {
    const int4 r = refs_at(c, p);
    count += used(p, r.x) + used(p + 1, r.y) + used(p + 2, r.z) + used(p + 3, r.w);
  }
  uint64_t total;
  block_scan(count, total, s_warp);
  const int live = (int)total;
  if (tid == 0 && live == c.num_pages) w.head[4] = live;
  int below = 0;  // live pages so far
  for (long base = 0; base < c.num_pages; base += 4 * SCAN) {
    count = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (base + q * SCAN >= c.num_pages) break;
      const int p = (int)base + q * SCAN + 4 * tid;
      count += (uint64_t)(used(p, f.r[q].x) + used(p + 1, f.r[q].y) + used(p + 2, f.r[q].z) + used(p + 3, f.r[q].w)) << (16 * q);
    }
    const uint64_t before = block_scan(count, total, s_warp);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (base + q * SCAN >= c.num_pages) break;
      int at = below + (int)(before >> (16 * q) & 0xffff);
      const int v[4] = {f.r[q].x, f.r[q].y, f.r[q].z, f.r[q].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = (int)base + q * SCAN + 4 * tid + e;
        const bool is = used(p, v[e]);
        if (p < c.num_pages) {
          if (p == live) w.head[4] = at;
          if (p < live && !is) w.list[p - at] = p;
          if (p >= live) w.rank[p] = is ? at : -1;
          if (p >= live && is) w.high[at] = p;
        }
        at += is;
      }
      below += (int)(total >> (16 * q) & 0xffff);
    }
    if (base + 4 * SCAN < c.num_pages) f = four_at(c, (int)base + 4 * SCAN);
  }
  __syncthreads();
  if (tid == 0) {
    w.head[0] = 1;
    w.head[3] = live;
    w.head[1] = live - w.head[4];
  }
}

// Copies of whole pages (codes and scales), a grid-stride loop over pieces of
// 16 KB: four 16-byte loads in flight per thread, six CTAs per SM.  155 MB of
// pages moved: 47 us, 6.6 TB/s read and written.
constexpr int COPY_THREADS = 256;
constexpr int COPY_PIECE = COPY_THREADS * 64;
template <class Pair>
__device__ __forceinline__ void copy_pages(const Cache& c, int copies, Pair pair) {
  const long bytes = c.page_bytes();
  const int pieces = (int)((bytes + COPY_PIECE - 1) / COPY_PIECE);
  const long all = (long)copies * pieces;
  for (long t = blockIdx.x; t < all; t += gridDim.x) {
    const int k = (int)(t / pieces), piece = (int)(t % pieces);
    int src, dst;
    pair(k, src, dst);
    const long at = (long)piece * COPY_PIECE;
    const uint4* s = reinterpret_cast<const uint4*>(c.codes + src * bytes + at);
    uint4* o = reinterpret_cast<uint4*>(c.codes + dst * bytes + at);
    const int m = (int)((min(bytes - at, (long)COPY_PIECE)) >> 4);
    uint4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((int)threadIdx.x + e * COPY_THREADS < m) x[e] = __ldcs(s + threadIdx.x + e * COPY_THREADS);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((int)threadIdx.x + e * COPY_THREADS < m) __stcs(o + threadIdx.x + e * COPY_THREADS, x[e]);
    if (piece == 0) {
      const int ns = c.page_scales();
      for (int e = threadIdx.x; e < ns; e += COPY_THREADS) c.scales[(long)dst * ns + e] = c.scales[(long)src * ns + e];
    }
  }
}

__global__ void __launch_bounds__(COPY_THREADS)
    resize_apply_kernel(Cache c, const int32_t* __restrict__ slots, const int32_t* __restrict__ lens, int n, Work w) {
  pdl_wait();
  if (w.head[0] == 0) return;
  const int lane = threadIdx.x & 31;
  // A slot's copied page shows in the lists: its destination is the first of the pages it wanted.
  for (int i = blockIdx.x * (COPY_THREADS / 32) + (threadIdx.x >> 5); i < n; i += gridDim.x * (COPY_THREADS / 32)) {
    const int slot = slots[i], new_len = lens[i], old_len = c.lens[slot];
    const int first = w.first[i], next = i + 1 < n ? w.first[i + 1] : w.head[2];
    const int have = c.pages_of(old_len), want = c.pages_of(new_len);
    const int copy = next - first - max(0, want - have);
    int32_t* row = c.table + (long)slot * c.max_pages;
    __syncwarp();
    if (lane == 0) {
      if (copy) {
        const int edge = min(old_len, new_len) >> c.ps_log2, page = w.list[first];
        atomicAdd(&c.refs[row[edge]], -1);
        row[edge] = page;
        c.refs[page] = 1;
      }
      c.lens[slot] = new_len;
    }
    for (int j = have + lane; j < want; j += 32) {
      const int page = w.list[first + copy + j - have];
      row[j] = page;
      c.refs[page] = 1;
    }
    for (int j = want + lane; j < have; j += 32) row[j] = -1;
  }
  copy_pages(c, w.head[1], [&](int k, int& src, int& dst) {
    src = w.copy[2 * k];
    dst = w.list[w.copy[2 * k + 1]];
  });
}

__global__ void __launch_bounds__(COPY_THREADS)
    fork_apply_kernel(Cache c, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n, Work w) {
  pdl_wait();
  if (w.head[0] == 0) return;
  const int lane = threadIdx.x & 31;
  for (int i = blockIdx.x * (COPY_THREADS / 32) + (threadIdx.x >> 5); i < n; i += gridDim.x * (COPY_THREADS / 32)) {
    const int len = c.lens[src[i]], whole = len >> c.ps_log2;
    const int32_t* from = c.table + (long)src[i] * c.max_pages;
    int32_t* to = c.table + (long)dst[i] * c.max_pages;
    for (int j = lane; j < whole; j += 32) {
      const int page = from[j];
      to[j] = page;
      if (c.page_ok(page))
        atomicAdd(&c.refs[page], 1);
      else
        set_device_err(DERR_KV8_TABLE);
    }
    if (lane == 0 && (len & (c.ps - 1))) {
      const int page = w.list[w.first[i]];
      to[whole] = page;
      c.refs[page] = 1;
    }
    if (lane == 0) c.lens[dst[i]] = len;
  }
  copy_pages(c, w.head[1], [&](int k, int& s, int& t) {
    s = w.copy[2 * k];
    t = w.list[w.copy[2 * k + 1]];
  });
}

__global__ void __launch_bounds__(COPY_THREADS) compact_apply_kernel(Cache c, int32_t* live_out, Work w) {
  pdl_wait();
  if (w.head[0] == 0) return;
  const int lane = threadIdx.x & 31, low = w.head[4], live = w.head[3], moves = w.head[1];
  const int stride = gridDim.x * COPY_THREADS, me = blockIdx.x * COPY_THREADS + threadIdx.x;
  for (int j = me; j < moves; j += stride) {
    const int from = w.high[low + j], to = w.list[j];
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
  }
  for (int i = me >> 5; i < c.num_slots; i += stride >> 5) {
    int32_t* row = c.table + (long)i * c.max_pages;
    const int len = c.len_of(i), used = len < 0 ? 0 : c.pages_of(len);
    if (len < 0) set_device_err(DERR_KV8_ARGS);
    for (int j = lane; j < used; j += 32) {
      const int page = row[j], r = !c.page_ok(page) ? -1 : page < live ? 0 : w.rank[page];
      if (r < 0)
        set_device_err(DERR_KV8_TABLE);
      else if (page >= live)
        row[j] = w.list[r - low];
    }
  }
  if (me == 0 && live_out) *live_out = live;
  copy_pages(c, moves, [&](int k, int& s, int& t) {
    s = w.high[low + k];
    t = w.list[k];
  });
}

// The apply kernel starts while the plan runs (programmatic dependent launch)
// and waits for it in pdl_wait().
template <class... P, class... A>
static inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                                       A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int APPLY_CTAS = 148 * 6;

static inline cudaError_t resize(const Cache& c, const int32_t* slots, const int32_t* lens, int n, void* work,
                                 cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  const Work w = work_of(work, n, c.num_pages);
  static DeviceOnce once;
  cudaError_t e = run_once_per_device(once, [] {
    return cudaFuncSetAttribute(resize_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                MAX_SLOTS / 8 + 8 + MAX_SEQS * 16);
  });
  if (e != cudaSuccess) return e;
  resize_plan_kernel<<<1, PLAN_THREADS, plan_smem(c, n, true), st>>>(c, slots, lens, n, w);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(resize_apply_kernel, dim3(APPLY_CTAS), COPY_THREADS, 0, st, c, slots, lens, n, w);
}
static inline cudaError_t fork(const Cache& c, const int32_t* src, const int32_t* dst, int n, void* work,
                               cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  const Work w = work_of(work, n, c.num_pages);
  fork_plan_kernel<<<1, PLAN_THREADS, plan_smem(c, n, false), st>>>(c, src, dst, n, w);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(fork_apply_kernel, dim3(APPLY_CTAS), COPY_THREADS, 0, st, c, src, dst, n, w);
}
static inline cudaError_t compact(const Cache& c, int32_t* live, void* work, cudaStream_t st) {
  const Work w = work_of(work, 0, c.num_pages);
  compact_plan_kernel<<<1, PLAN_THREADS, 0, st>>>(c, w);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(compact_apply_kernel, dim3(APPLY_CTAS), COPY_THREADS, 0, st, c, live, w);
}

}  // namespace kv8

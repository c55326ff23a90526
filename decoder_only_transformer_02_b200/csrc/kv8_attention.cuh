// Causal attention over the paged 8-bit cache.
//
// Sequence i of the call has len cached tokens, the last q_i = cu[i+1] - cu[i]
// of which are the call's rows; the row at position p sees the tokens 0..p.
// Query head j reads key/value head j / group, group = n_head / n_kv_head.
//   s_t = (q . kc_t) ks_t / sqrt(d)      kc, vc codes; ks, vs their blocks' scales
//   p_t = exp(s_t - max)                 lse = max + log(sum p_t)
//   o   = sum_t p_t vs_t vc_t / sum_t p_t
//
// For single tokens (and up to tens of rows per key/value head) the codes of
// the cache are the traffic, 2 d bytes per token and head: the kernel streams
// them once.
//  - S^T = K Q^T and O^T = V^T P^T on mma m16n8k16 (f16 in, fp32 out), tokens
//    (then dimensions) in the 16 rows and 8 query rows in the columns: with few
//    rows this wastes half as much of an instruction as rows in the 16 would.
//    (tcgen05 could have tokens in its 64 or more rows and 8 query rows in the
//    columns too, but takes the tokens' operand from shared memory: the converted
//    codes would be stored there and read once more.)
//  - A thread's 16 bytes of a key are its A operand: which dimension stands at
//    which k index is free as long as Q agrees, so no code moves between lanes.
//    The values' operand pairs two tokens of one dimension, a byte permute.
//  - Codes become f16 exactly: e4m3 by its conversion instruction, int8 by
//    placing the byte under 1024's exponent and subtracting 1152.  Q's rows are
//    scaled by a power of two into f16's range (bf16 has fewer fraction bits,
//    so this too is exact for components within 2^-29 of the row's largest).
//  - Weights: p vs 2^6 / vref in f16 (2^-11 relative), vref the largest value
//    scale up to the token, so that they stay below 2^14; sums, maxima, scores and O in fp32.
//  - The row maximum moves only when a score passes it by 2^8 (one vote per
//    step instead of a reduction over the lanes).
//  - Each warp keeps three 4 KB steps of codes in flight (asynchronous copies
//    into a ring of its own).  Loading the next step into registers instead
//    kept a third as many bytes in flight: 131 us where this took 118 (32
//    sequences of up to 16384 tokens, 705 MB; 116.5 by now, 6.1 TB/s of 6.56 measured).
//  - All sequences' 16-token groups, tile after tile (a tile: the rows of one
//    sequence and key/value head), are one line of work that is cut into equal
//    parts, one per CTA; a part's warps take its steps in turn.  A tile
//    that was cut leaves partial results that a second kernel joins in order,
//    so the result is the same in every run.
#pragma once
#include "kv8.cuh"

namespace kv8 {

constexpr int GROUP = 16;  // tokens of a step: one page, one matrix instruction's rows

// ------------------------------------------------------------- instructions
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transpose of an 8 x 8 matrix of 16-bit elements held as mma fragments
__device__ __forceinline__ uint32_t mat_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// four codes to two f16 pairs
template <int FMT>
__device__ __forceinline__ void codes_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == GPT2_KV_E4M3) {
    lo = e4m3x2_to_half2(w & 0xffffu);
    hi = e4m3x2_to_half2(w >> 16);
  } else {
    const uint32_t u = w ^ 0x80808080u;  // code + 128
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));  // 1152
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  }
}
// asynchronous copy of 16 bytes to shared memory; zeros where `on` is false (the address must be valid all the same)
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// ------------------------------------------------------------- the work line
struct Join;
struct Call {
  Cache c;
  int layer, H, group, n, rows, max_q;
  const bf16* q;
  long ldq;
  bf16* out;
  long ldo;
  float* lse;
  const int32_t *slots, *cu;
  Join* join;         // [grid]
  float* part;        // [grid][2][rows of a tile][d + 2]
  int narrow;         // most rows per key/value head of a sequence that the streaming kernel takes
  int setup;          // units of the line that beginning a tile counts
  int min_part;       // fewest units of a CTA's part
  uint32_t zero;      // 0
};

struct Entry {
  int slot, len, a, q;  // q = 0: nothing to do
};
// tiles of a sequence: kvh for every row_tile rows of (token, head of the group)
__device__ __forceinline__ int row_tiles(const Call& k, int q, int row_tile) {
  return (int)(((long)q * k.group + row_tile - 1) / row_tile);
}
__device__ __forceinline__ int groups_of(int len) { return (len + GROUP - 1) / GROUP; }

// A tile takes its 16-token groups and `setup` units more on the line, what
// beginning one costs in groups.
struct Line {
  long long* pre;  // [n + 1] units before each sequence
  int4* entry;     // [n] Entry
  int setup;
  static __host__ __device__ size_t bytes(int n) { return (size_t)n * 16 + (size_t)(n + 1) * 8; }
  __device__ Line(void* smem, int n, int setup_)
      : pre(reinterpret_cast<long long*>(static_cast<int4*>(smem) + n)), entry(static_cast<int4*>(smem)), setup(setup_) {}
};

// Fills the line; false when the offsets are bad (the call is refused).
__device__ __forceinline__ bool lay_out(const Call& k, int row_tile, const Line& line, long long* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const bool report = blockIdx.x == 0;
  long long base = 0;
  bool bad = false;
  for (int i0 = 0; i0 < k.n; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    long long x = 0;
    if (i < k.n) {
      const int a = k.cu[i], b = k.cu[i + 1], slot = k.slots[i];
      bad |= a < 0 || b < a || b > k.rows;
      int q = b - a, len = 0;
      if (q > 0) {
        len = k.c.len_of(slot);
        if (len < q || q > k.max_q) {
          q = 0;
          if (report) set_device_err(DERR_KV8_ARGS);
        } else if ((long)q * k.group <= k.narrow) {
          x = (long long)k.c.kvh * row_tiles(k, q, row_tile) * (groups_of(len) + line.setup);
        }
      }
      line.entry[i] = make_int4(slot, len, a, q);
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
    if (i < k.n) line.pre[i] = before + x - own;
    __syncthreads();
  }
  if (threadIdx.x == 0) line.pre[k.n] = base;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && report) set_device_err(DERR_KV8_ARGS);
    return false;
  }
  return true;
}

struct Piece {
  Entry e;
  int head, row0, g0, g1, groups;  // key/value head, first row, groups [g0, g1) of `groups`
  long long next;                  // where the line goes on
};
// the tile that holds unit `at` of the line, and its groups up to `end`
__device__ __forceinline__ Piece piece_at(const Call& k, const Line& line, int row_tile, long long at, long long end) {
  int lo = 0, hi = k.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (line.pre[mid] <= at) lo = mid; else hi = mid;
  }
  Piece p;
  const int4 e = line.entry[lo];
  p.e.slot = e.x, p.e.len = e.y, p.e.a = e.z, p.e.q = e.w;
  p.groups = groups_of(p.e.len);
  const int size = p.groups + line.setup;
  const long long rel = at - line.pre[lo];
  const int tile = (int)(rel / size);
  const int u = (int)(rel - (long long)tile * size);
  p.next = min(at - u + size, end);
  p.g0 = max(0, u - line.setup);
  p.g1 = max(0, (int)(p.next - at) + u - line.setup);
  p.head = tile % k.c.kvh;
  p.row0 = (tile / k.c.kvh) * row_tile;
  return p;
}

// What is left to join: the tile that begins in part x and goes on in the next
// parts (parts = 0: none).  Written by every CTA for its own x.
struct Join {
  int parts, tile_rows, row0, head, a, pad[3];
};

// --------------------------------------------------------- streaming kernel
constexpr int STAGES = 3;  // steps in flight per warp

// CTAs of four warps per SM: as many as their registers and rings allow
__host__ __device__ constexpr int ctas_of(int rt, int d) { return rt * d <= 512 ? 4 : rt * d <= 1024 ? 3 : 2; }

template <int D, int NT, int W>
struct Shape {
  static constexpr int RT = 8 * NT;               // rows of a tile
  static constexpr int CH = D / 64;               // 16-byte pieces of a key per thread
  static constexpr int U = D == 64 ? 2 : 1;      // groups per step
  static constexpr int VW = D / 32;               // 4-byte words of a value per thread and token
  static constexpr int SIDE = GROUP * D;          // bytes of a group's keys, or values
  static constexpr int STEP = 2 * U * SIDE;       // 4 KB
  static constexpr int WARP = STAGES * STEP + (STAGES * U * 8 + 127) / 128 * 128;  // a warp's ring: codes, groups' scales
  static constexpr int OUT = W * RT * (D + 2) * 4;
  static constexpr int BYTES = W * WARP > OUT ? W * WARP : OUT;  // the results reuse the rings
  static_assert(WARP % 16 == 0 && BYTES % 16 == 0, "16-byte copies and the work line's entries");
  static constexpr int CTAS = W > 4 ? 1 : ctas_of(RT, D);
};

// The codes go through a ring of asynchronous copies, private to each warp.
// Shared memory holds token sigma(i) of a group in row i, sigma exchanging the
// last two of each four, and 16-byte piece j of a row at place j ^ (row & 7) of
// its 128 bytes (d = 128), or j ^ (row / 2 & 3) of its 64 (d = 64).  Then the
// key loads (row g, pieces CH tg ..) and the value loads (rows 2 tg, pieces of
// dimension D/8 g) of every eight (16-byte) or sixteen (8-byte) lanes fall into
// different banks.
template <int D>
__device__ __forceinline__ int place(int row, int piece) {
  return D == 128 ? row * 128 + ((piece ^ (row & 7)) << 4) : row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}
// the row of token t of a group, and the token of a row
__device__ __forceinline__ int sigma(int t) { return t ^ ((t >> 1) & 1); }

// MANY: sequences may have several rows, some of which do not see all tokens of
// a tile.  (With single rows that part of the loop, never taken, costs 0.3 us of
// 6.4 for one sequence and 0.6 of 19.2 for 64: its instructions are fetched.)
template <int FMT, int D, int NT, int W, bool SPLIT, bool MANY>
__global__ void __launch_bounds__(32 * W, (Shape<D, NT, W>::CTAS)) stream_kernel(const Call k) {
  using S = Shape<D, NT, W>;
  constexpr int RT = S::RT, CH = S::CH, U = S::U, VW = S::VW;
  extern __shared__ __align__(128) uint8_t s_dyn[];
  __shared__ long long s_warp[W];
  float* s_o = reinterpret_cast<float*>(s_dyn);      // [W][RT][D], after the rings
  float* s_m = s_o + W * RT * D;                     // [W][RT]
  float* s_l = s_m + W * RT;
  const Line line(s_dyn + S::BYTES, k.n, k.setup);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tg = lane & 3;
  const Cache& c = k.c;
  long long at = 0, end = 1, per = 1;
  int join_parts = 0;
  Piece p;
  int first_page = 0;
  if (SPLIT) {
    pdl_launch();
    const bool ok = lay_out(k, RT, line, s_warp);
    const long long total = ok ? line.pre[k.n] : 0;
    per = max((long long)k.min_part, (total + gridDim.x - 1) / gridDim.x);
    at = blockIdx.x * per;
    end = min(total, at + per);
  } else {
    // CTA (x, y): tile x of sequence y
    const int i = blockIdx.y;
    bool bad = false;
    for (int j = threadIdx.x; j < k.n; j += 32 * W) bad |= k.cu[j] < 0 || k.cu[j + 1] < k.cu[j] || k.cu[j + 1] > k.rows;
    p.e.slot = k.slots[i];
    p.e.a = k.cu[i];
    p.e.q = k.cu[i + 1] - p.e.a;
    // (the page ids are requested with the length, not behind it)
    if ((unsigned)p.e.slot < (unsigned)c.num_slots)
      first_page = c.table[(long)p.e.slot * c.max_pages + min(((lane / U * W + warp) * U + lane % U) >> (c.ps_log2 - 4), c.max_pages - 1)];
    p.e.len = c.len_of(p.e.slot);
    p.head = blockIdx.x % c.kvh;
    p.row0 = blockIdx.x / c.kvh * RT;
    p.g0 = 0;
    p.g1 = p.groups = groups_of(p.e.len);
    p.next = 1;
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0) set_device_err(DERR_KV8_ARGS);
      at = end;
    } else if (p.e.q <= 0 || (long)p.row0 >= (long)p.e.q * k.group) {
      at = end;
    } else if (p.e.len < p.e.q || p.e.q > k.max_q) {
      if (threadIdx.x == 0) set_device_err(DERR_KV8_ARGS);
      at = end;
    } else if ((long)p.e.q * k.group > k.narrow) {
      at = end;
    }
  }
  const float sl2 = LOG2E_F * (D == 64 ? 0.125f : 0.08838834764831845f);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_dyn) + warp * S::WARP;
  // copies: lane x takes piece x % (D / 16) of rows x / (D / 16), + 32 / (D / 16), ...
  constexpr int PER_ROW = D / 16, ROWS = 32 / PER_ROW;
  const int crow = lane / PER_ROW, cpiece = lane % PER_ROW;

  while (at < end) {
    if (SPLIT) {
      p = piece_at(k, line, RT, at, end);
      if (p.g0 == 0 && p.g1 > 0 && p.g1 < p.groups) {
        join_parts = (int)((p.next + p.groups - p.g1 - 1) / per) - blockIdx.x + 1;
        if (threadIdx.x == 0) {
          Join j;
          j.parts = join_parts, j.tile_rows = min(RT, p.e.q * k.group - p.row0), j.row0 = p.row0, j.head = p.head, j.a = p.e.a;
          k.join[blockIdx.x] = j;
        }
      }
    }
    at = p.next;
    if (SPLIT && p.g1 == p.g0) continue;  // only the tile's setup units are in this part
    const int tile_rows = min(RT, p.e.q * k.group - p.row0);

    // ---- this warp's steps: the groups g0 + (W k + warp) U .. + U - 1, k = 0, 1, ..., and their pages
    const int own = p.g0 + warp * U;
    const int32_t* table = c.table + (long)p.e.slot * c.max_pages;
    const int gp_log2 = c.ps_log2 - 4;  // groups of a page
    const long page_stride = c.page_bytes();
    const uint8_t* head_base = c.codes + ((long)k.layer * 2 * c.kvh + p.head) * c.ps * D;
    const long side_stride = (long)c.kvh * c.ps * D;
    int pg = 0, base = 0;
    float ksc = 0.f, vsc = 0.f;
    auto batch = [&](int from, bool known) {  // lane x: page and scales of group x % U of step from + x / U
      base = from;
      const int gi = own + (from + lane / U) * (W * U) + lane % U;
      pg = 0;
      ksc = vsc = 0.f;
      if (gi < p.g1) {
        pg = known ? first_page : table[gi >> gp_log2];
        if (c.page_ok(pg)) {
          ksc = c.scales[c.unit(pg, k.layer, 0, p.head)];
          vsc = c.scales[c.unit(pg, k.layer, 1, p.head)];
          if (!(vsc <= 3.0e38f)) ksc = vsc;  // a block that is not a number is none for the scores either
        } else {
          set_device_err(DERR_KV8_TABLE);
          pg = -1;
          ksc = vsc = __uint_as_float(NAN_SCALE);
        }
      }
    };
    // starts the copies of a step; keys and values of tokens behind the last become zero, and those of a page
    // outside the pool (what would be read in its place may be no numbers, which a weight of 0 does not hide)
    auto load = [&](int step, int stage) {
      const int gi = own + step * (W * U), at = (step - base) * U;
      const uint32_t dst = ring + stage * S::STEP;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int page = __shfl_sync(0xffffffffu, pg, at + u);
        const uint8_t* t = head_base + max(page, 0) * page_stride + (((gi + u) << 4) & (c.ps - 1)) * D;
        const int left = gi + u < p.g1 && page >= 0 ? p.e.len - (gi + u) * GROUP : 0;
#pragma unroll
        for (int r = 0; r < GROUP; r += ROWS) {
          const int row = r + crow, tok = sigma(row);
          const uint32_t o = dst + 2 * u * S::SIDE + place<D>(row, cpiece);
          const uint8_t* src = t + (tok * D + cpiece * 16);
          copy_async16(o, src, tok < left);
          copy_async16(o + S::SIDE, src + side_stride, tok < left);
        }
      }
      copy_commit();
      // (the scales come behind the codes' requests: they may still be on their way)
      const float a = __shfl_sync(0xffffffffu, ksc, (at + lane) & 31);
      const float b = __shfl_sync(0xffffffffu, vsc, (at + lane) & 31);
      if (lane < U)
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ring + STAGES * S::STEP + 8 * (stage * U + lane)), "f"(a), "f"(b)
                     : "memory");
    };
    float o[D / 16][NT][4], m[NT][2], mu[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      mu[nt][0] = mu[nt][1] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    }
    // vref: the largest value scale so far (not of NaN blocks).  A row's weights
    // have to be held relative to what the row sees, or a later token's value could
    // leave nothing of them: batches count the groups that every row sees, the
    // others follow one by one.  (Rows that do not see the group that raises it
    // have only O scaled, in fp32.)
    float vref = 0.f, vinv = 0.f;
    auto raise = [&](float top) {  // (the warp's lanes agree)
      if (top > vref) {
        if (vref > 0.f) {
          const float f = vref / top;
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[mt][nt][e] *= f;
        }
        vref = top;
        vinv = 1.f / top;
      }
    };
    auto raise_batch = [&](int minpos) {  // the groups that begin at minpos, the first row's token, or before
      const int gi = own + (base + lane / U) * (W * U) + lane % U;
      const bool on = gi * GROUP <= minpos && vsc <= 3.0e38f;
      raise(__uint_as_float(__reduce_max_sync(0xffffffffu, on ? __float_as_uint(vsc) : 0u)));
    };
    batch(0, !SPLIT);
#pragma unroll
    for (int st = 0; st < STAGES - 1; ++st) {
      if (own + st * (W * U) < p.g1) load(st, st);
      else copy_commit();
    }

    // ---- Q: row g of each n tile; this thread's dimensions as those of its key pieces
    uint32_t qb[NT][CH][8];
    float rowf[NT][2];  // score factor of rows 2 tg, 2 tg + 1
    const int pos0 = p.e.len - p.e.q, minpos = pos0 + p.row0 / k.group;
    int pos[NT][2];     // the last token they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = p.row0 + nt * 8 + g;
      const bool on = nt * 8 + g < tile_rows;
      const int tok = on ? r / k.group : 0;
      const bf16* src = k.q + (long)(p.e.a + tok) * k.ldq + (p.head * k.group + (on ? r - tok * k.group : 0)) * D + 16 * CH * tg;
      uint32_t raw[CH][8], mx = 0;
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (on) {
          x = *reinterpret_cast<const uint4*>(src + 16 * ch);
          y = *reinterpret_cast<const uint4*>(src + 16 * ch + 8);
        }
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          raw[ch][e] = w[e];
          mx = __vmaxu2(mx, w[e] & 0x7fff7fffu);
        }
      }
      mx = max(mx & 0xffffu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // times 2^(14 - exponent of the largest), at most 2^126
      const int E = max((int)(mx >> 7), 15);
      const float up = __uint_as_float((uint32_t)(268 - E) << 23), down = __uint_as_float((uint32_t)(E - 14) << 23);
#pragma unroll
      for (int ch = 0; ch < CH; ++ch)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = unpack_bf16x2(raw[ch][e]);
          qb[nt][ch][e] = half2_of(f.x * up, f.y * up);
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        rowf[nt][j] = __shfl_sync(0xffffffffu, down, 8 * tg + 4 * j) * sl2;
        pos[nt][j] = pos0 + (p.row0 + nt * 8 + 2 * tg + j) / k.group;
      }
    }
    raise_batch(minpos);

    int stage = 0;
    for (int step = 0, gi = own; gi < p.g1; ++step, gi += W * U) {
      copy_wait<STAGES - 2>();
      __syncwarp();  // every lane's copies have landed, and the stage before is free
      {
        const int nx = step + STAGES - 1, free_stage = stage == 0 ? STAGES - 1 : stage - 1;
        if (own + nx * (W * U) < p.g1) {
          if (nx - base >= 32 / U) {
            batch(nx, false);
            load(nx, free_stage);
            raise_batch(minpos);
          } else {
            load(nx, free_stage);
          }
        } else {
          copy_commit();
        }
      }
      const uint32_t buf = ring + stage * S::STEP, sc = ring + STAGES * S::STEP + 8 * stage * U;
      stage = stage == STAGES - 1 ? 0 : stage + 1;
      // ---- scores
      float s[U][NT][4], vs[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float ks;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs[u]) : "r"(sc + 8 * u));
        vs[u] = vs[u] * vinv * 64.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.f;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          const uint4 x = lds128(buf + 2 * u * S::SIDE + place<D>(g, CH * tg + ch));
          const uint4 y = lds128(buf + 2 * u * S::SIDE + place<D>(g + 8, CH * tg + ch));
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            codes_half<FMT>(xs[w], a0, a2);
            codes_half<FMT>(ys[w], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(s[u][nt], a0, a1, a2, a3, qb[nt][ch][2 * w], qb[nt][ch][2 * w + 1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float f0 = ks * rowf[nt][0], f1 = ks * rowf[nt][1];
          s[u][nt][0] *= f0;
          s[u][nt][1] *= f1;
          s[u][nt][2] *= f0;
          s[u][nt][3] *= f1;
        }
      }
      const int t0 = gi * GROUP;
      const bool edge = t0 + U * GROUP - 1 > minpos || gi + U > p.g1;
      if (edge) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gi + u >= p.g1 || t0 + u * GROUP + sigma(g) + 8 * (e >> 1) > pos[nt][e & 1]) s[u][nt][e] = -INFINITY;
      }
      // ---- row maxima, moved only past 2^8
      float top[NT][2];
      bool past = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
          for (int u = 1; u < U; ++u) x = fmaxf(x, fmaxf(s[u][nt][j], s[u][nt][j + 2]));
          top[nt][j] = x;
          past |= x > m[nt][j] + 8.f;
        }
      if (__any_sync(0xffffffffu, past)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float al[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = top[nt][j];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float nm = fmaxf(m[nt][j], x);
            al[j] = m[nt][j] == -INFINITY ? 0.f : ex2_approx(m[nt][j] - nm);
            m[nt][j] = nm;
            mu[nt][j] = nm == -INFINITY ? 0.f : nm;
            l[nt][j] *= al[j];
          }
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            o[mt][nt][0] *= al[0];
            o[mt][nt][1] *= al[1];
            o[mt][nt][2] *= al[0];
            o[mt][nt][3] *= al[1];
          }
        }
      }
      // ---- weights, and the values' products
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (MANY && edge) {
          float v;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(sc + 8 * u + 4));
          if (v <= 3.0e38f) {
            raise(v);
            vs[u] = v * vinv * 64.f;
          }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = ex2_approx(s[u][nt][e] - mu[nt][e & 1]);
            l[nt][e & 1] += x;
            w[e] = x * vs[u];
            if (edge && s[u][nt][e] == -INFINITY) w[e] = 0.f;  // also where the scale is NaN
          }
          pb[nt][0] = mat_trans(half2_of(w[0], w[1]));
          pb[nt][1] = mat_trans(half2_of(w[2], w[3]));
        }
        uint32_t vc[4][VW];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 2 * tg + (e & 1) + 8 * (e >> 1);
          const uint32_t a = buf + (2 * u + 1) * S::SIDE;
          if (D == 64) {
            const uint2 x = lds64(a + place<D>(row, g >> 1) + 8 * (g & 1));
            vc[e][0] = x.x, vc[e][1] = x.y;
          } else {
            const uint4 x = lds128(a + place<D>(row, g));
            vc[e][0] = x.x, vc[e][1] = x.y, vc[e][VW - 2] = x.z, vc[e][VW - 1] = x.w;
          }
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          uint32_t a0, a1, a2, a3;
          const int sel = mt & 1 ? 0x7362 : 0x5140;
          codes_half<FMT>(__byte_perm(vc[0][mt >> 1], vc[1][mt >> 1], sel), a0, a1);
          codes_half<FMT>(__byte_perm(vc[2][mt >> 1], vc[3][mt >> 1], sel), a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[mt][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        }
      }
    }
    // ---- the warps' results joined in shared memory
    copy_wait<0>();
    __syncthreads();  // every ring is done with
    const float unit = vref * (1.f / 64.f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[nt][j];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int r = nt * 8 + 2 * tg + j;
        if (g == 0) {
          s_m[warp * RT + r] = m[nt][j];
          s_l[warp * RT + r] = x;
        }
        float* dst = s_o + (warp * RT + r) * D + (D / 8) * g;
#pragma unroll
        for (int mt = 0; mt < D / 16; mt += 2)
          *reinterpret_cast<float4*>(dst + 2 * mt) =
              make_float4(o[mt][nt][j] * unit, o[mt][nt][j + 2] * unit, o[mt + 1][nt][j] * unit, o[mt + 1][nt][j + 2] * unit);
      }
    __syncthreads();
    const bool whole = !SPLIT || (p.g0 == 0 && p.g1 == p.groups);
    float* part = k.part + ((long)blockIdx.x * 2 + (p.g0 == 0)) * RT * (D + 2);
    for (int i = threadIdx.x; i < tile_rows * (D / 4); i += 32 * W) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      float M = s_m[r], L = 0.f;
#pragma unroll
      for (int w = 1; w < W; ++w) M = fmaxf(M, s_m[w * RT + r]);
      const float Mu = M == -INFINITY ? 0.f : M;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = ex2_approx(s_m[w * RT + r] - Mu);
        const float4 x = *reinterpret_cast<const float4*>(s_o + (w * RT + r) * D + 4 * d4);
        L += f * s_l[w * RT + r];
        a.x += f * x.x, a.y += f * x.y, a.z += f * x.z, a.w += f * x.w;
      }
      if (whole) {
        const float inv = 1.f / L;
        const int row = p.row0 + r, tok = row / k.group, h = p.head * k.group + row - tok * k.group;
        *reinterpret_cast<uint2*>(k.out + (long)(p.e.a + tok) * k.ldo + h * D + 4 * d4) =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        if (d4 == 0 && k.lse) k.lse[(long)(p.e.a + tok) * k.H + h] = (M + log2f(L)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4*>(part + r * D + 4 * d4) = a;
        if (d4 == 0) {
          part[RT * D + r] = M;
          part[RT * D + RT + r] = L;
        }
      }
    }
    __syncthreads();
  }
  if (SPLIT && join_parts == 0 && threadIdx.x == 0) k.join[blockIdx.x].parts = 0;
  pdl_wait();  // (behind the wide kernel: this one does not end before it)
}

// CTAs (x, ...) join the tile that began in part x of the line and went on past
// it: its partial results lie with part x (place 1) and the parts after it
// (place 0).  The warps take the parts in turn; results meet in warp order.
// A tile's rows are spread over the CTAs of y, four or fewer each: 32 rows cut into
// 37 parts, 17.0 us for the whole call where one CTA for all rows took 36.7.
constexpr int J_WARPS = 8;
__host__ __device__ constexpr int join_ctas(int rt) { return rt / 4; }
template <int D, int RT>
__device__ __forceinline__ void join_tile(const Call& k, const Join* join, const float* part, int part_x, int cta_y) {
  constexpr int LANES = D / 4;  // threads of a row
  __shared__ float4 s_a[J_WARPS][32];
  __shared__ float s_m[J_WARPS][32], s_l[J_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Join t = join[part_x];
  if (t.parts == 0) return;
  constexpr long SIZE = (long)RT * (D + 2);
  const float* first = part + ((long)part_x * 2 + 1) * SIZE;
  for (int r0 = cta_y * (32 / LANES); r0 < t.tile_rows; r0 += join_ctas(RT) * (32 / LANES)) {
    const int r = r0 + lane / LANES, d4 = lane % LANES;
    const bool on = r < t.tile_rows;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
#pragma unroll 4
      for (int j = warp; j < t.parts; j += J_WARPS) {
        const float* src = first + (j ? (2 * j - 1) * SIZE : 0);
        const float m = src[RT * D + r], l = src[RT * D + RT + r];
        const float4 x = *reinterpret_cast<const float4*>(src + r * D + 4 * d4);
        const float nm = fmaxf(M, m), nu = nm == -INFINITY ? 0.f : nm;
        const float f = ex2_approx(M - nu), h = ex2_approx(m - nu);
        M = nm;
        L = L * f + l * h;
        a.x = a.x * f + x.x * h, a.y = a.y * f + x.y * h, a.z = a.z * f + x.z * h, a.w = a.w * f + x.w * h;
      }
    }
    s_a[warp][lane] = a;
    s_m[warp][lane] = M;
    s_l[warp][lane] = L;
    __syncthreads();
    if (warp == 0 && on) {
      const int nw = min(t.parts, J_WARPS);
      for (int w = 1; w < nw; ++w) M = fmaxf(M, s_m[w][lane]);
      const float Mu = M == -INFINITY ? 0.f : M;
      L = 0.f;
      a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < nw; ++w) {
        const float f = ex2_approx(s_m[w][lane] - Mu);
        const float4 x = s_a[w][lane];
        L += f * s_l[w][lane];
        a.x += f * x.x, a.y += f * x.y, a.z += f * x.z, a.w += f * x.w;
      }
      const float inv = 1.f / L;
      const int row = t.row0 + r, tok = row / k.group, h = t.head * k.group + row - tok * k.group;
      *reinterpret_cast<uint2*>(k.out + (long)(t.a + tok) * k.ldo + h * D + 4 * d4) =
          make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
      if (d4 == 0 && k.lse) k.lse[(long)(t.a + tok) * k.H + h] = (M + log2f(L)) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}
template <int D, int RT>
__global__ void __launch_bounds__(32 * J_WARPS) join_kernel(const Call k) {
  pdl_wait();
  join_tile<D, RT>(k, k.join, k.part, blockIdx.x, blockIdx.y);
}

static inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n > 0 ? n : 148;
}

// Sequences with more rows per key/value head than this go to the tensor-core
// kernel of kv8_prompt.cuh.  64 rows here and 65 there, d = 64: 16 sequences of
// 4096 93 and 103 us, 64 of 1024 110 and 146; d = 128: 181 and 166, 209 and 211.
// Twice as many rows cost here twice as much (32 rows: 55 and 61 us; 102 and 114),
// there next to nothing (96 rows: 104 and 148; 170 and 216).
constexpr int NARROW_ROWS = 64;
static inline long narrow_rows(long rows) { return rows < NARROW_ROWS ? rows : NARROW_ROWS; }

// rows of a tile in a call with more than NARROW_ROWS
__host__ __device__ constexpr int wide_row_tile(int d) { return d == 128 ? 16 : 32; }
// rows of a tile: the call's rows per key/value head, 8 to 32 (16 at d = 128)
static inline int row_tile_of(const Cache& c, int group, int max_q) {
  const long r = narrow_rows((long)group * max_q);
  return r <= 8 ? 8 : r <= 16 ? 16 : wide_row_tile(c.d);
}
static inline int parts_of(const Cache& c, int rt) {
  return sm_count() * ctas_of(rt, c.d);
}

static inline size_t stream_workspace_bytes(const Cache& c, int H, int max_q) {
  const int rt = row_tile_of(c, H / c.kvh, max_q);
  return (size_t)parts_of(c, rt) * (sizeof(Join) + 2 * rt * (c.d + 2) * 4);
}

template <int FMT, int D, int NT, int W, bool SPLIT, bool MANY>
static inline cudaError_t stream_launch(const Call& k, void* work, cudaStream_t st, bool behind) {
  using S = Shape<D, NT, W>;
  const size_t smem = S::BYTES + (SPLIT ? Line::bytes(k.n) : 0);
  static DeviceOnce once;
  cudaError_t e = run_once_per_device(once, [] {
    return cudaFuncSetAttribute(stream_kernel<FMT, D, NT, W, SPLIT, MANY>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                S::BYTES + (SPLIT ? (int)Line::bytes(MAX_SEQS) : 0));
  });
  if (e != cudaSuccess) return e;
  Call a = k;
  if (!SPLIT) {
    const long tiles = (long)k.c.kvh * ((narrow_rows((long)k.max_q * k.group) + S::RT - 1) / S::RT);
    const dim3 grid((unsigned)tiles, k.n);
    if (behind) return launch_after(stream_kernel<FMT, D, NT, W, SPLIT, MANY>, grid, 32 * W, smem, st, a);
    stream_kernel<FMT, D, NT, W, SPLIT, MANY><<<grid, 32 * W, smem, st>>>(a);
    return cudaGetLastError();
  }
  const int grid = parts_of(k.c, S::RT);
  a.join = static_cast<Join*>(work);
  a.part = reinterpret_cast<float*>(a.join + grid);
  if (behind) {
    e = launch_after(stream_kernel<FMT, D, NT, W, SPLIT, MANY>, dim3(grid), 32 * W, smem, st, a);
  } else {
    stream_kernel<FMT, D, NT, W, SPLIT, MANY><<<grid, 32 * W, smem, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || behind) return e;  // (the wide kernel's join takes these tiles too)
  return launch_after(join_kernel<D, S::RT>, dim3(grid, join_ctas(S::RT)), 32 * J_WARPS, 0, st, a);
}
// Where no slot can hold more than this, every tile is one CTA's: no line, no
// join.  Sequences of 1024, whole and cut into parts: one 6.8 and 8.0 us, 8 7.4 and
// 10.1, 64 25.2 and 29.4; of 2032: 10.2 and 8.5, 11.4 and 13.1, 42.6 and 46.4; of
// 4080: 16.7 and 9.6, 18.9 and 19.5, 76.9 and 77.9.  d = 128, 8 heads, 1024: 10.5
// and 9.5, 10.6 and 11.9, 32.9 and 34.3; 2032: 16.2 and 10.3, 17.9 and 16.1, 57.7 and
// 52.9.  (One sequence alone would want the parts from 1300 tokens on, at d = 128
// from 900; it goes by the table's width, since the lengths are on the device.)
// One sequence of 777: 6.4 with eight warps, sixteen 7.2.
constexpr long WHOLE_TOKENS = 2048;
static inline bool whole_tiles(const Cache& c) { return (long)c.max_pages * c.ps <= WHOLE_TOKENS; }
template <int FMT, int D, int NT, bool MANY>
static inline cudaError_t stream_mode(const Call& k, void* work, cudaStream_t st, bool behind) {
  const long tiles = (long)k.n * k.c.kvh * ((narrow_rows((long)k.max_q * k.group) + 8 * NT - 1) / (8 * NT));
  if (whole_tiles(k.c))
    return tiles <= sm_count() ? stream_launch<FMT, D, NT, 8, false, MANY>(k, work, st, behind) : stream_launch<FMT, D, NT, 4, false, MANY>(k, work, st, behind);
  return stream_launch<FMT, D, NT, 4, true, MANY>(k, work, st, behind);
}
template <int FMT, int D, int NT>
static inline cudaError_t stream_many(const Call& k, void* work, cudaStream_t st, bool behind) {
  return k.max_q > 1 ? stream_mode<FMT, D, NT, true>(k, work, st, behind) : stream_mode<FMT, D, NT, false>(k, work, st, behind);
}
template <int FMT>
static inline cudaError_t stream_rows(const Call& k, void* work, cudaStream_t st, bool behind) {
  const int rt = behind ? wide_row_tile(k.c.d) : row_tile_of(k.c, k.group, k.max_q);  // (as the join behind both has it)
  if (k.c.d == 64)
    return rt == 8 ? stream_many<FMT, 64, 1>(k, work, st, behind) : rt == 16 ? stream_many<FMT, 64, 2>(k, work, st, behind) : stream_many<FMT, 64, 4>(k, work, st, behind);
  return rt == 8 ? stream_many<FMT, 128, 1>(k, work, st, behind) : stream_many<FMT, 128, 2>(k, work, st, behind);
}

// behind: it follows the wide kernel of the same call and may start before that one ends
static inline cudaError_t stream(Call k, void* work, cudaStream_t st, bool behind) {
  k.setup = k.c.d == 64 ? 16 : 4;
  k.min_part = k.setup + 8;
  return k.c.fmt == GPT2_KV_INT8 ? stream_rows<GPT2_KV_INT8>(k, work, st, behind) : stream_rows<GPT2_KV_E4M3>(k, work, st, behind);
}

}  // namespace kv8

// Causal attention over the paged 8-bit cache.
//
// Sequence i of the call has len cached tokens, the last q_i = cu[i+1] - cu[i]
// of which are the call's rows; the row at position p sees the tokens 0..p.
// Query head j reads key/value head j / (n_head / n_kv_head).
//   s_t = (q . kc_t) ks_t / sqrt(d)      kc, vc codes; ks, vs their pages' scales
//   p_t = exp(s_t - max)                 lse = max + log(sum p_t)
//   o   = sum_t p_t vs_t vc_t / sum_t p_t
#pragma once
#include "kv8.cuh"

namespace kv8 {

// One warp per (row, query head): 32 tokens at a time, one score per lane,
// then the values with the lanes over the head's dimensions.
template <int FMT, int D>
__global__ void __launch_bounds__(128)
    attention_kernel(Cache c, int layer, const bf16* __restrict__ q, long ldq, bf16* __restrict__ out, long ldo,
                     float* __restrict__ lse, int H, const int32_t* __restrict__ slots, const int32_t* __restrict__ cu,
                     int n, int rows, int max_q) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= cu[i] < 0 || cu[i + 1] < cu[i] || cu[i + 1] > rows;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_device_err(DERR_KV8_ARGS);
    return;
  }
  const long id = ((long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (id >= (long)rows * H) return;
  const int row = (int)(id / H), h = (int)(id % H);
  if (row < cu[0] || row >= cu[n]) return;
  int lo = 0, hi = n;  // the sequence with cu[lo] <= row < cu[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= row) lo = mid; else hi = mid;
  }
  const int a = cu[lo], b = cu[lo + 1], slot = slots[lo];
  const int len = c.len_of(slot);
  if (a > row || b <= row || len < b - a || b - a > max_q) {
    if (lane == 0) set_device_err(DERR_KV8_ARGS);
    return;
  }
  const int kvh = h / (H / c.kvh), last = len - (b - row);  // position of this row
  const float sc = LOG2E_F / sqrtf((float)D);
  float qv[D];
#pragma unroll
  for (int e = 0; e < D; ++e) qv[e] = bf2f(q[row * ldq + h * D + e]);
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  for (int t0 = 0; t0 <= last; t0 += 32) {
    const int t = t0 + lane;
    float s = -INFINITY, vs = 0.f;
    long vu = 0;
    bool ok = true;
    if (t <= last) {
      const int page = c.table[(long)slot * c.max_pages + (t >> c.ps_log2)];
      ok = c.page_ok(page);
      if (ok) {
        const long ku = c.unit(page, layer, 0, kvh);
        vu = c.unit(page, layer, 1, kvh);
        const uint32_t* kr = reinterpret_cast<const uint32_t*>(c.codes + ku * c.tile() + (long)(t & (c.ps - 1)) * D);
        float acc = 0.f;
#pragma unroll
        for (int e = 0; e < D / 4; ++e) {
          float f[4];
          unpack4<FMT>(kr[e], f);
#pragma unroll
          for (int g = 0; g < 4; ++g) acc = fmaf(f[g], qv[4 * e + g], acc);
        }
        s = acc * c.scales[ku] * sc;
        vs = c.scales[vu];
      }
    }
    if (__any_sync(0xffffffffu, !ok)) {
      if (lane == 0) set_device_err(DERR_KV8_TABLE);
      return;
    }
    const float nm = fmaxf(m, warp_max(s)), alpha = exp2f(m - nm), p = t <= last ? exp2f(s - nm) : 0.f;
    m = nm;
    l = l * alpha + warp_sum(p);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] *= alpha;
    const int cnt = min(32, last + 1 - t0);
    for (int j = 0; j < cnt; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p * vs, j);
      const long u = __shfl_sync(0xffffffffu, vu, j);
      const uint8_t* vr = c.codes + u * c.tile() + (long)((t0 + j) & (c.ps - 1)) * D;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        float f[4];
        unpack4<FMT>(vr[e * 32 + lane], f);
        o[e] = fmaf(pj, f[0], o[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) out[row * ldo + h * D + e * 32 + lane] = f2bf(o[e] / l);
  if (lane == 0 && lse) lse[(long)row * H + h] = (m + log2f(l)) * 0.6931471805599453f;
}

static inline size_t attention_workspace_bytes(const Cache&, int, int, int, int) { return 256; }

static inline cudaError_t attention(const Cache& c, int layer, const bf16* q, long ldq, bf16* out, long ldo,
                                    float* lse, int H, const int32_t* slots, const int32_t* cu, int n, int rows,
                                    int max_q, void* work, cudaStream_t st) {
  (void)work;
  if (n == 0 || rows == 0) return cudaSuccess;
  const unsigned grid = (unsigned)(((long)rows * H + 3) / 4);
#define KV8_GO(F, D_) attention_kernel<F, D_><<<grid, 128, 0, st>>>(c, layer, q, ldq, out, ldo, lse, H, slots, cu, n, rows, max_q)
  if (c.fmt == GPT2_KV_INT8)
    c.d == 64 ? KV8_GO(GPT2_KV_INT8, 64) : KV8_GO(GPT2_KV_INT8, 128);
  else
    c.d == 64 ? KV8_GO(GPT2_KV_E4M3, 64) : KV8_GO(GPT2_KV_E4M3, 128);
#undef KV8_GO
  return cudaGetLastError();
}

}  // namespace kv8

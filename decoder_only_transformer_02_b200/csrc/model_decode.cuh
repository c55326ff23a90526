// Generation: the forward pass one token at a time with a KV cache, and an
// on-device top-k sampler ("Let's reproduce GPT-2 (124M)", Chapters:
// sampling init, prefix tokens; sampling loop).
//
// A prefill runs the training forward on the prefix [B, T0] and copies every
// layer's keys and values into the cache; each decode step then takes one new
// token per sequence at the next position, computes its 12 layers with M = B
// rows (the tcgen05 GEMMs, a one-query attention over the cached keys), the
// lm_head logits [B, Vp] and the next token.  bf16 mode only.
//
// Sampling rule (the pages name a sampling loop but no rule): top-k sampling
// from softmax(logits / temperature) over the k largest logits of the real
// vocabulary [0, V), ties at the k-th place to the lower id; k = 1 or
// temperature 0 is the greedy argmax.  The uniform u of row b for the token at
// position p is the top 53 bits of splitmix64(seed * 2^32 + p * 2^16 + b)
// (Steele, Lea and Flood's generator), so a CPU restatement draws the same u.
//
// The same on a paged 8-bit cache that the caller owns (gpt2_kv8_prefill,
// gpt2_kv8_decode_step): sequences of different lengths, each row at its own
// slot's next position; keys and values are rounded into the cache and the
// attention reads it.
#pragma once
#include "kv8_prompt.cuh"
#include "model_pass.cuh"

namespace gen {

constexpr int SAMPLE_THREADS = 1024;
constexpr int MAX_TOP_K = 64;

// x[b] = wte[tok[b]] + wpe[pos] (fp32), pos_of[b] instead of pos where given; ids outside [0, Vp) flag the error
// word and embed as wpe only
__global__ void embed_kernel(const int32_t* __restrict__ tok, const float* __restrict__ wte,
                             const float* __restrict__ wpe, float* __restrict__ x, int B, int C, int Vp, int pos,
                             const int32_t* __restrict__ pos_of, int* __restrict__ bad) {
  const int c4 = C / 4;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < B * c4; i += gridDim.x * blockDim.x) {
    const int b = i / c4, c = i % c4;
    const int id = tok[b];
    float4 p = reinterpret_cast<const float4*>(wpe + (long)(pos_of ? pos_of[b] : pos) * C)[c];
    if (id >= 0 && id < Vp) {
      const float4 w = reinterpret_cast<const float4*>(wte + (long)id * C)[c];
      p.x += w.x;
      p.y += w.y;
      p.z += w.z;
      p.w += w.w;
    } else if (c == 0) {
      atomicExch(bad, 1);
    }
    reinterpret_cast<float4*>(x + (long)b * C)[c] = p;
  }
}

// kv[b][t][0:C] = k, kv[b][t][C:2C] = v of rows b*T0 + t of one layer's qkv
// [B*T0, 3C] (t < T0), 16 bytes per thread
__global__ void fill_cache_kernel(const bf16* __restrict__ qkv, bf16* __restrict__ kv, int B, int T0, int C,
                                  int P) {
  const int c8 = 2 * C / 8;  // 16-byte chunks of k and v
  const long n = (long)B * T0 * c8;
  for (long i = blockIdx.x * (long)blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x) {
    const long r = i / c8;
    const int c = (int)(i % c8);
    const int b = (int)(r / T0), t = (int)(r % T0);
    const uint4 v = reinterpret_cast<const uint4*>(qkv + r * 3L * C + C)[c];
    reinterpret_cast<uint4*>(kv + ((long)b * P + t) * 2L * C)[c] = v;
  }
}

// One query per (sequence, head) against the cached keys 0..pos: stores the
// new key and value at pos, then o = softmax(q k^T / sqrt(d)) v with the
// scores in shared memory and fixed-order reductions.  qkv [B, 3C], kv layer
// base [max_B][P][2C], out [B, C].  Dynamic shared memory: (pos+1) floats.
__global__ void __launch_bounds__(256) attn_kernel(const bf16* __restrict__ qkv, bf16* __restrict__ kv,
                                                   bf16* __restrict__ out, int H, int P, int pos, float sl2) {
  extern __shared__ float sc[];
  __shared__ float qs[64];
  __shared__ float red[256];
  const int b = blockIdx.x / H, h = blockIdx.x % H;
  const int C = H * 64;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bf16* row = qkv + (long)b * 3 * C;
  bf16* cache = kv + (long)b * P * 2 * C;
  if (tid < 16) {
    // the new key (threads 0-7) and value (8-15) at position pos
    const int part = tid >> 3, c = tid & 7;
    reinterpret_cast<uint4*>(cache + (long)pos * 2 * C + part * C + h * 64)[c] =
        reinterpret_cast<const uint4*>(row + (1 + part) * C + h * 64)[c];
  }
  if (tid < 64) qs[tid] = bf2f(row[h * 64 + tid]);
  __syncthreads();
  // scores in log2 units
  float mx = -INFINITY;
  for (int t = tid; t <= pos; t += 256) {
    const uint4* kr = reinterpret_cast<const uint4*>(cache + (long)t * 2 * C + h * 64);
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 u = kr[c];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack_bf16x2(w[e]);
        s = fmaf(qs[8 * c + 2 * e], f.x, fmaf(qs[8 * c + 2 * e + 1], f.y, s));
      }
    }
    s *= sl2;
    sc[t] = s;
    mx = fmaxf(mx, s);
  }
  red[tid] = mx;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) red[tid] = fmaxf(red[tid], red[tid + o]);
    __syncthreads();
  }
  mx = red[0];
  __syncthreads();
  float sum = 0.f;
  for (int t = tid; t <= pos; t += 256) {
    const float e = exp2f(sc[t] - mx);
    sc[t] = e;
    sum += e;
  }
  red[tid] = sum;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) red[tid] += red[tid + o];
    __syncthreads();
  }
  const float inv = 1.f / red[0];
  __syncthreads();
  // o[d] = sum_t p_t v_t[d]: thread (slice, d) takes the keys t = slice mod 4
  const int d = tid & 63, sl = tid >> 6;
  float acc = 0.f;
  for (int t = sl; t <= pos; t += 4) acc = fmaf(sc[t], bf2f(cache[(long)t * 2 * C + C + h * 64 + d]), acc);
  red[tid] = acc;
  __syncthreads();
  if (tid < 64) {
    const float o = ((red[d] + red[64 + d]) + red[128 + d]) + red[192 + d];
    out[(long)b * C + h * 64 + d] = f2bf(o * inv);
  }
  (void)lane;
  (void)warp;
}

__device__ __forceinline__ uint64_t sm64(uint64_t x) {
  x += 0x9E3779B97F4A7C15ull;
  x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
  x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
  return x ^ (x >> 31);
}

// (v, i) precedes (w, j) in the sampler's order: larger logit first, lower id on ties
__device__ __forceinline__ bool before(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

// One CTA per sequence: the next token from its logits row z (bf16 [Vp],
// row stride ld) over ids [0, V).  k rounds each find the next element in
// (logit desc, id asc) order; p_i = exp((z_i - z_top) / temperature) in
// double, inverse CDF at u.  top_k <= 1 or temperature <= 0: argmax.  The
// draw's position and sequence are pos_next and the row, or pos_of[row] + 1 and
// seq_of[row] where given.
__global__ void __launch_bounds__(SAMPLE_THREADS) sample_kernel(const bf16* __restrict__ z, long ld, int V,
                                                               float temperature, int top_k, uint64_t seed,
                                                               int pos_next, const int32_t* __restrict__ pos_of,
                                                               const int32_t* __restrict__ seq_of,
                                                               int32_t* __restrict__ next) {
  __shared__ float bv[SAMPLE_THREADS / 32];
  __shared__ int bi[SAMPLE_THREADS / 32];
  __shared__ float top_v[MAX_TOP_K];
  __shared__ int top_i[MAX_TOP_K];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bf16* zr = z + (long)b * ld;
  const int k = (top_k <= 1 || temperature <= 0.f) ? 1 : min(top_k, min(V, MAX_TOP_K));
  float pv = INFINITY;  // previous selection (the order starts above every logit)
  int pi = -1;
  for (int r = 0; r < k; ++r) {
    float v = -INFINITY;
    int i = 0x7fffffff;
    for (int j = tid; j < V; j += SAMPLE_THREADS) {
      const float x = bf2f(zr[j]);
      if (before(pv, pi, x, j) && before(x, j, v, i)) {
        v = x;
        i = j;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, v, o);
      const int oi = __shfl_xor_sync(0xffffffffu, i, o);
      if (before(ov, oi, v, i)) {
        v = ov;
        i = oi;
      }
    }
    if (lane == 0) {
      bv[warp] = v;
      bi[warp] = i;
    }
    __syncthreads();
    v = bv[0];
    i = bi[0];
    for (int w = 1; w < SAMPLE_THREADS / 32; ++w)
      if (before(bv[w], bi[w], v, i)) {
        v = bv[w];
        i = bi[w];
      }
    if (tid == 0) {
      top_v[r] = v;
      top_i[r] = i;
    }
    pv = v;
    pi = i;
    __syncthreads();
  }
  if (tid == 0) {
    int pick = top_i[0];
    if (k > 1) {
      double p[MAX_TOP_K], tot = 0.0;
      for (int r = 0; r < k; ++r) {
        p[r] = exp(((double)top_v[r] - (double)top_v[0]) / (double)temperature);
        tot += p[r];
      }
      const int p_next = pos_of ? pos_of[b] + 1 : pos_next, seq = seq_of ? seq_of[b] : b;
      const uint64_t key = ((seed & 0xFFFFFFFFull) << 32) | ((uint64_t)(p_next & 0xFFFF) << 16) | (uint64_t)(seq & 0xFFFF);
      const double u = (double)(sm64(key) >> 11) * (1.0 / 9007199254740992.0);
      double c = 0.0;
      pick = top_i[k - 1];
      for (int r = 0; r < k; ++r) {
        c += p[r];
        if (c / tot > u) {
          pick = top_i[r];
          break;
        }
      }
    }
    next[b] = pick;
  }
}

// Before a paged step's resize: row b's token goes to the slot's position
// lens[slot], or, for a prefill, T0 <= P tokens to 0 .. T0 - 1.  A slot or length
// out of range, or without room (P positions), asks for the length -1, which
// refuses the call, and so does every slot of a prefill whose freeing resize
// was refused (freed, the word that a resize leaves in its workspace).  The
// position is in 0 .. P - 1 in any case: the embedding reads it.
__global__ void paged_before_kernel(kv8::Cache c, const int32_t* __restrict__ slots, int P, int B, int T0,
                                    const int32_t* __restrict__ freed, int32_t* __restrict__ pos,
                                    int32_t* __restrict__ new_len) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  const int len = T0 > 0 ? T0 - 1 : c.len_of(slots[b]);  // -1: out of range
  const bool ok = len >= 0 && len < P && (T0 <= 0 || *freed != 0);
  pos[b] = ok ? len : 0;
  new_len[b] = ok ? len + 1 : -1;
}
// After it: the row offsets of append and attention, all 0 (no rows) when the
// resize was refused (resized, its word), so that the cache stays as it was.
// (The lengths do not tell: slots of a refused prefill may hold T0 tokens already.)
__global__ void paged_after_kernel(int B, int rows, const int32_t* __restrict__ resized, int32_t* __restrict__ cu) {
  const bool ok = *resized != 0;
  for (int b = threadIdx.x; b <= B; b += blockDim.x) cu[b] = ok ? b * rows : 0;
}

}  // namespace gen

static int gen_alloc(gpt2* h) {
  const long mb = h->maxB, C = h->C;
  if (h->dec_logits != nullptr) return GPT2_OK;
#define GEN_ALLOC(ptr, bytes) \
  if ((ptr) == nullptr) ALLOC(h, ptr, bytes)
  GEN_ALLOC(h->dec_x, (size_t)mb * C * 4);
  GEN_ALLOC(h->dec_mean, (size_t)mb * 4);
  GEN_ALLOC(h->dec_rstd, (size_t)mb * 4);
  GEN_ALLOC(h->dec_ln, (size_t)mb * C * 2);
  GEN_ALLOC(h->dec_qkv, (size_t)mb * 3 * C * 2);
  GEN_ALLOC(h->dec_att, (size_t)mb * C * 2);
  GEN_ALLOC(h->dec_u, (size_t)mb * 4 * C * 2);
  GEN_ALLOC(h->dec_a, (size_t)mb * 4 * C * 2);
  GEN_ALLOC(h->pg_pos, (size_t)mb * 4);
  GEN_ALLOC(h->pg_len, (size_t)mb * 4);
  GEN_ALLOC(h->pg_cu, (size_t)(mb + 1) * 4);
  GEN_ALLOC(h->dec_logits, (size_t)mb * h->Vp * 2);
#undef GEN_ALLOC
  return GPT2_OK;
}
// the dense cache of gpt2_prefill / gpt2_decode_step
static int gen_alloc_dense(gpt2* h) {
  if (h->kv == nullptr) ALLOC(h, h->kv, (size_t)h->L * h->maxB * h->P * 2 * h->C * 2);
  return GPT2_OK;
}

static int gen_check(gpt2* h, float temperature, int top_k, int32_t* d_next) {
  if (h->prec != GPT2_BF16) return set_err(h, GPT2_EINVAL, "generation needs bf16 mode");
  if (d_next == nullptr) return set_err(h, GPT2_EINVAL, "next-token pointer is NULL");
  if (top_k < 1 || top_k > gen::MAX_TOP_K || !(temperature >= 0.f))
    return set_err(h, GPT2_EINVAL, "top_k must lie in [1, 64] and temperature must be >= 0");
  return gen_alloc(h);
}

static int gen_sample(gpt2* h, const bf16* rows, long ld, int B, float temperature, int top_k, uint64_t seed,
                      int pos_next, const int32_t* pos_of, const int32_t* seq_of, int32_t* d_next) {
  gen::sample_kernel<<<B, gen::SAMPLE_THREADS, 0, h->stream>>>(rows, ld, h->V, temperature, top_k, seed, pos_next,
                                                              pos_of, seq_of, d_next);
  LAUNCH_CHECK(h);
  h->dec_rows = B;
  return GPT2_OK;
}

// the last position's logits of every sequence: rows b*T0 + T0-1
static int gen_last_logits(gpt2* h, int B, int T0) {
  CU_CHECK(h, cudaMemcpy2DAsync(h->dec_logits, (size_t)h->Vp * 2, (const bf16*)h->logits + (size_t)(T0 - 1) * h->Vp,
                                (size_t)T0 * h->Vp * 2, (size_t)h->Vp * 2, B, cudaMemcpyDeviceToDevice, h->stream));
  return GPT2_OK;
}

// Prefill: the training forward on [B, T0] (logits only), every layer's keys
// and values into the cache, the last position's logits kept and sampled.
static int prefill_impl(gpt2* h, const int32_t* tok, int B, int T0, float temperature, int top_k, uint64_t seed,
                        int32_t* d_next) {
  RET_IF(gen_check(h, temperature, top_k, d_next));
  if (T0 > h->P) return set_err(h, GPT2_EINVAL, "prefix longer than block_size");
  RET_IF(gen_alloc_dense(h));
  RET_IF(forward_impl(h, tok, nullptr, B, T0, false, 1.f));
  const int C = h->C;
  Views w{h};
  for (int l = 0; l < h->L; ++l) {
    const long n = (long)B * T0 * (2 * C / 8);
    gen::fill_cache_kernel<<<grid_for(n, 256), 256, 0, h->stream>>>(
        (const bf16*)w.qkv(l), h->kv + (size_t)l * h->maxB * h->P * 2 * C, B, T0, C, h->P);
    LAUNCH_CHECK(h);
  }
  RET_IF(gen_last_logits(h, B, T0));
  RET_IF(gen_sample(h, h->dec_logits, h->Vp, B, temperature, top_k, seed, T0, nullptr, nullptr, d_next));
  h->gen_B = B;
  h->gen_len = T0;
  return GPT2_OK;
}

// The layers of one decode step on the rows of dec_x [B, C], and the logits;
// attend(layer) turns dec_qkv into dec_att.
template <class Attend>
static int decode_layers(gpt2* h, int B, Attend attend) {
  const int C = h->C, L = h->L;
  for (int l = 0; l < L; ++l) {
    const LayerOffsets& o = h->lo[l];
    RET_IF(op_ln_fwd(h, h->dec_x, o.ln1g, o.ln1b, h->dec_ln, h->dec_mean, h->dec_rstd, B));
    RET_IF(op_lin_fwd(h, h->dec_ln, B, C, o.attnw, 3 * C, o.attnb, LIN_PLAIN, h->dec_qkv, nullptr, nullptr));
    RET_IF(attend(l));
    RET_IF(op_lin_fwd(h, h->dec_att, B, C, o.projw, C, o.projb, LIN_RESID, h->dec_x, nullptr, h->dec_x));
    RET_IF(op_ln_fwd(h, h->dec_x, o.ln2g, o.ln2b, h->dec_ln, h->dec_mean, h->dec_rstd, B));
    RET_IF(op_lin_fwd(h, h->dec_ln, B, C, o.fcw, 4 * C, o.fcb, LIN_GELU, h->dec_u, h->dec_a, nullptr));
    RET_IF(op_lin_fwd(h, h->dec_a, B, 4 * C, o.mpw, C, o.mpb, LIN_RESID, h->dec_x, nullptr, h->dec_x));
  }
  RET_IF(op_ln_fwd(h, h->dec_x, h->lnfg, h->lnfb, h->dec_ln, h->dec_mean, h->dec_rstd, B));
  return op_lin_fwd(h, h->dec_ln, B, C, h->wte, h->Vp, NO_OFF, LIN_NOBIAS, h->dec_logits, nullptr, nullptr);
}

// One decode step: tokens [B] at position pos (= the number of positions the
// cache holds), all layers with M = B, logits [B, Vp], the next token.
static int decode_impl(gpt2* h, const int32_t* tok, int B, int pos, float temperature, int top_k, uint64_t seed,
                       int32_t* d_next) {
  RET_IF(gen_check(h, temperature, top_k, d_next));
  if (tok == nullptr) return set_err(h, GPT2_EINVAL, "tokens pointer is NULL");
  if (B != h->gen_B || B < 1) return set_err(h, GPT2_ESTATE, "decode needs a prefill with the same batch first");
  if (pos != h->gen_len) return set_err(h, GPT2_ESTATE, "decode position must follow the cached positions");
  if (pos >= h->P) return set_err(h, GPT2_EINVAL, "position reaches block_size");
  const int C = h->C;
  {
    KTimer kt(h, KC_EMB, 0.0, 8.0 * B * C);
    gen::embed_kernel<<<grid_for((long)B * C / 4, 256), 256, 0, h->stream>>>(
        tok, h->P32(h->wte), h->P32(h->wpe), h->dec_x, B, C, h->Vp, pos, nullptr, h->d_bad);
    LAUNCH_CHECK(h);
  }
  const float sl2 = 1.4426950408889634f / sqrtf((float)(C / h->H));
  RET_IF(decode_layers(h, B, [&](int l) -> int {
    KTimer kt(h, KC_ATTN_F, 4.0 * B * (pos + 1.0) * C, 0.0);
    gen::attn_kernel<<<B * h->H, 256, (size_t)(pos + 1) * 4, h->stream>>>(
        h->dec_qkv, h->kv + (size_t)l * h->maxB * h->P * 2 * C, h->dec_att, h->H, h->P, pos, sl2);
    LAUNCH_CHECK(h);
    return GPT2_OK;
  }));
  RET_IF(gen_sample(h, h->dec_logits, h->Vp, B, temperature, top_k, seed, pos + 1, nullptr, nullptr, d_next));
  h->gen_len = pos + 1;
  return GPT2_OK;
}

// ------------------------------------------------ on a paged 8-bit cache
// Scratch of the cache calls, for max_B rows.  A larger pool needs more: a new
// block, at least twice the old one's size so that there are few of them; the
// old one stays until the handle is destroyed, since graphs captured with it
// may be replayed.
static int paged_scratch(gpt2* h, const kv8::Cache& c) {
  const int B = h->maxB < kv8::MAX_SEQS ? h->maxB : kv8::MAX_SEQS;
  const size_t a = kv8::workspace_bytes(B, c.num_pages), b = kv8::attention_workspace_bytes(c, h->H, B, B, 1);
  const size_t need = a > b ? a : b;
  if (need <= h->pg_work_bytes) return GPT2_OK;
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(h->stream, &capturing) != cudaSuccess) cudaGetLastError();
  if (capturing != cudaStreamCaptureStatusNone)
    return set_err(h, GPT2_ESTATE, "a larger cache than before needs a call outside the capture first");
  int k = 0;
  while (h->pg_old[k] != nullptr) ++k;
  uint8_t* p = nullptr;
  const size_t bytes = need > 2 * h->pg_work_bytes ? need : 2 * h->pg_work_bytes;
  ALLOC(h, p, bytes);
  h->pg_old[k] = h->pg_work;
  h->pg_work = p;
  h->pg_work_bytes = bytes;
  return GPT2_OK;
}

// Checks of both calls.
static int paged_check(gpt2* h, const gpt2_kv8* cache, kv8::Cache& c, const int32_t* slots, const int32_t* tok, int B,
                       float temperature, int top_k, int32_t* d_next) {
  RET_IF(gen_check(h, temperature, top_k, d_next));
  if (slots == nullptr || tok == nullptr) return set_err(h, GPT2_EINVAL, "slots or tokens pointer is NULL");
  if (B < 1 || B > h->maxB) return set_err(h, GPT2_EINVAL, "B out of range");
  if (!kv8::cache_of(cache, c)) return set_err(h, GPT2_EINVAL, "the cache's sizes or pointers are out of their limits");
  if (c.L != h->L || c.kvh != h->H || c.d != h->C / h->H)
    return set_err(h, GPT2_EINVAL, "the cache has other layers, heads or head dimension than the model");
  if (B > kv8::MAX_SEQS) return set_err(h, GPT2_EINVAL, "more rows than a cache call takes");
  return paged_scratch(h, c);
}

// The slots' lengths for T0 new tokens from position 0 (T0 > 0: behind the
// resize that freed them) or one more, and the row offsets (none when refused).
static int paged_room(gpt2* h, const kv8::Cache& c, const int32_t* slots, int B, int T0) {
  const int32_t* go = kv8::go_word(h->pg_work);
  gen::paged_before_kernel<<<(B + 255) / 256, 256, 0, h->stream>>>(c, slots, h->P, B, T0, go, h->pg_pos, h->pg_len);
  LAUNCH_CHECK(h);
  CU_CHECK(h, kv8::resize(c, slots, h->pg_len, B, h->pg_work, h->stream));
  h->launches += 2;
  gen::paged_after_kernel<<<1, 256, 0, h->stream>>>(B, T0 > 0 ? T0 : 1, go, h->pg_cu);
  LAUNCH_CHECK(h);
  return GPT2_OK;
}

static int paged_prefill_impl(gpt2* h, const gpt2_kv8* cache, const int32_t* slots, const int32_t* tok, int B, int T0,
                              float temperature, int top_k, uint64_t seed, int32_t* d_next) {
  kv8::Cache c;
  RET_IF(paged_check(h, cache, c, slots, tok, B, temperature, top_k, d_next));
  if (T0 > h->P) return set_err(h, GPT2_EINVAL, "prefix longer than block_size");
  RET_IF(forward_impl(h, tok, nullptr, B, T0, false, 1.f));
  // free the slots, then take T0 tokens each
  CU_CHECK(h, cudaMemsetAsync(h->pg_len, 0, (size_t)B * 4, h->stream));
  CU_CHECK(h, kv8::resize(c, slots, h->pg_len, B, h->pg_work, h->stream));
  h->launches += 2;
  RET_IF(paged_room(h, c, slots, B, T0));
  Views w{h};
  const int C = h->C;
  for (int l = 0; l < h->L; ++l) {
    const bf16* qkv = (const bf16*)w.qkv(l);
    CU_CHECK(h, kv8::append(c, l, qkv + C, qkv + 2 * C, 3L * C, slots, h->pg_cu, B, B * T0, h->stream));
    h->launches++;
  }
  RET_IF(gen_last_logits(h, B, T0));
  return gen_sample(h, h->dec_logits, h->Vp, B, temperature, top_k, seed, T0, h->pg_pos, slots, d_next);
}

static int paged_decode_impl(gpt2* h, const gpt2_kv8* cache, const int32_t* slots, const int32_t* tok, int B,
                             float temperature, int top_k, uint64_t seed, int32_t* d_next) {
  kv8::Cache c;
  RET_IF(paged_check(h, cache, c, slots, tok, B, temperature, top_k, d_next));
  const int C = h->C;
  RET_IF(paged_room(h, c, slots, B, 0));
  {
    KTimer kt(h, KC_EMB, 0.0, 8.0 * B * C);
    gen::embed_kernel<<<grid_for((long)B * C / 4, 256), 256, 0, h->stream>>>(
        tok, h->P32(h->wte), h->P32(h->wpe), h->dec_x, B, C, h->Vp, 0, h->pg_pos, h->d_bad);
    LAUNCH_CHECK(h);
  }
  RET_IF(decode_layers(h, B, [&](int l) -> int {
    KTimer kt(h, KC_ATTN_F, 0.0, 0.0);  // (the lengths are on the device)
    CU_CHECK(h, kv8::append(c, l, h->dec_qkv + C, h->dec_qkv + 2 * C, 3L * C, slots, h->pg_cu, B, B, h->stream));
    CU_CHECK(h, kv8::attention(c, l, h->dec_qkv, 3L * C, h->dec_att, C, nullptr, h->H, slots, h->pg_cu, B, B, 1, h->pg_work,
                               h->stream));
    h->launches += kv8::whole_tiles(c) ? 2 : 3;  // (whole tiles need no join)
    return GPT2_OK;
  }));
  return gen_sample(h, h->dec_logits, h->Vp, B, temperature, top_k, seed, 0, h->pg_pos, slots, d_next);
}

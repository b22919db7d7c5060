// Writing and reading back the 8-bit paged KV cache: awq_kv_append (rotation,
// quantization, placement) and awq_kv_dequant.
//
// Mathematics. Row i of sequence b has position p = len_b - n_b + i. K (and
// q) turn in the plane of each channel pair by the angle whose cosine and
// sine the table holds for p; V is taken as it is. The 16 tokens of an
// aligned block share one fp32 scale per head:
//   s  = max(max|x| over the block's new tokens / R, s_old, 2^-60)
//   c  = round(x / s),   R = 127 (int8) or 448 (e4m3)
// with s_old only where the block holds earlier tokens of the sequence; if
// that makes s grow, their codes become round(c_old s_old / s). x, maxima
// and scales are fp32, and the quotients are rounded as the real numbers they
// are: 16-bit values over the block's largest fall on the border between two
// codes often enough (one in 10^4 or so) that a reciprocal's error would show
// in the cache (0.0006 against 0.0002 of an e4m3 cache's values, in the
// 2-norm), so a product that comes near a border is settled by its remainder.
//
// What bounds it: HBM bytes for prompts, launch and load latency for single
// tokens. Hence one CTA per touched block of 16 tokens (so that a scale and
// its codes have one writer and no atomics) with the heads spread over
// blockIdx.y when there are few blocks; the block's table rows are read once
// into shared memory and used for every head; a warp holds a head's whole
// block in registers (one read of K and V: the maximum and the codes come
// from the same values).

#include "awq_kv.cuh"

namespace awq {
namespace kv {
namespace {

__device__ uint32_t g_kv_append_error = 0;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct AppendParams {
  Batch batch;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const float* rope;      // [rope_rows][rot]: cosines, then sines
  int64_t rope_stride;
  int32_t rope_rows, rot;
  int32_t interleaved;
  uint8_t* pages[2];      // K, V
  float* scales[2];
  int64_t page_stride, scale_stride;
  int32_t n_q_heads, n_kv_heads;
};

// Blocks of 16 positions that the last n tokens of a sequence touch.
__device__ __forceinline__ int touched(const Seq& s) {
  const int p0 = max(s.past, 0);
  return s.len > p0 ? (s.len - 1) / kBlock - p0 / kBlock + 1 : 0;
}

// x: channels 8l .. 8l+7 of a row, l the lane's place in the row's lanes.
// cs: the row's cosines and sines in shared memory.
template <int LPR>
__device__ __forceinline__ void rotate8(float (&x)[8], int l, const float* cs, int rot, bool interleaved) {
  const int half = rot >> 1;
  const int d0 = 8 * l;
  if (interleaved) {
    if (d0 < rot) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float c = cs[(d0 >> 1) + j], s = cs[half + (d0 >> 1) + j];
        const float a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = a * c - b * s;
        x[2 * j + 1] = b * c + a * s;
      }
    }
    return;
  }
  // the partner channels are half a rotation width away, in another lane
  const bool low = d0 < half, in = d0 < rot;
  const int lane = threadIdx.x & 31;
  const int src = in ? (low ? lane + (half >> 3) : lane - (half >> 3)) : lane;
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], src);
  if (in) {
    const float* c = cs + (low ? d0 : d0 - half);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = low ? x[j] * c[j] - y[j] * c[half + j] : x[j] * c[j] + y[j] * c[half + j];
  }
}

// x / s (x = hi + lo) rounded to odd in fp32: cut off, with the last bit set
// where anything was cut, so that rounding it to a code rounds the quotient
// itself. inv is 1 / s; the remainder fma(-q, s, hi) is exact.
__device__ __forceinline__ float quotient_odd(float hi, float lo, float s, float inv) {
  float q = hi * inv;
  if (q == 0.0f) return q;   // keeps its sign
  q = fmaf(fmaf(-q, s, hi), inv, q);
  const float r = fmaf(-q, s, hi) + lo;
  uint32_t bits = __float_as_uint(q);
  if (r != 0.0f) bits = (bits - ((r < 0.0f) != (q < 0.0f) ? 1u : 0u)) | 1u;
  return __uint_as_float(bits);
}

// Whether t, a quotient within 3 ulp, may lie on the other side of a border
// between two codes.
template <int FMT>
__device__ __forceinline__ bool near_border(float t) {
  if (FMT == AWQ_KV_INT8) return fabsf(t - rintf(t)) > 0.4999f;   // 127 * 3 * 2^-24 < 10^-4
  const uint32_t a = __float_as_uint(t) & 0x7fffffffu;
  // normal codes: the 20 bits that go are near their middle; subnormal ones (below 2^-6): always looked at
  return ((a - 0x7fff8u) & 0xfffffu) <= 16u || a - 1u < 0x3c7fffffu;
}

// The codes of eight values over the scale s.
template <int FMT>
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], float s, float inv) {
  float t[8];
  bool near = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    t[j] = x[j] * inv;
    near |= near_border<FMT>(t[j]);
  }
  if (near) {
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = quotient_odd(x[j], 0.0f, s, inv);
  }
  return make_uint2(Code<FMT>::encode4(t), Code<FMT>::encode4(t + 4));
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 8;            // lanes per row of a head
  constexpr int RPP = 32 / LPR;         // rows per warp pass
  constexpr int PASSES = kBlock / RPP;
  __shared__ int64_t scratch[40];
  __shared__ __align__(16) float cs[kBlock * D];
  pdl_launch();
  pdl_wait();

  int64_t rest;
  const int64_t slot = blockIdx.x;
  const int b = locate(
      p.batch.n_seqs, scratch, [&](int i) { return int64_t(touched(load_seq(p.batch, i, &g_kv_append_error))); },
      [&](int64_t) { return slot; }, &rest, static_cast<int64_t*>(nullptr));
  if (b < 0) return;
  const Seq s = load_seq(p.batch, b, &g_kv_append_error);
  const int p0 = max(s.past, 0);                       // first position written
  const int base = (p0 / kBlock + int(rest)) * kBlock;   // the block's first position
  const int lo = max(base, p0) - base;                 // tokens lo .. hi-1 of the block are new
  int hi = min(base + kBlock, s.len) - base;
  if (p.rope && base + hi > p.rope_rows) {              // positions that the table does not hold
    if (threadIdx.x == 0) atomicOr(&g_kv_append_error, kErrRange);
    hi = max(p.rope_rows - base, lo);
  }
  if (hi <= lo) return;
  // The loads that depend on nothing but the sequence go out together: the page's id, the table's rows, the first
  // task's keys or values.
  const int id = p.batch.table[int64_t(b) * p.batch.table_stride + base / p.batch.page_size];
  const int t0 = s.t0 + (base - s.past);               // row of the block's token 0 (may lie before t0)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LPR, sub = lane / LPR;
  const int workers = gridDim.y * kWarps, me = blockIdx.y * kWarps + warp;
  const int tasks = 2 * p.n_kv_heads;
  uint4 raw[PASSES];
  auto fetch = [&](int task) {                          // K or V rows of one head, zeros around the new ones
    const int which = task >= p.n_kv_heads;
    const int64_t stride = which ? p.v_stride : p.k_stride;
    const uint16_t* src = (which ? p.v : p.k) + int64_t(t0) * stride + (which ? task - p.n_kv_heads : task) * D + 8 * l;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + sub;
      raw[i] = r >= lo && r < hi ? *reinterpret_cast<const uint4*>(src + r * stride) : make_uint4(0, 0, 0, 0);
    }
  };
  if (me < tasks) fetch(me);
  if (p.rope) {
    for (int r = lo + warp; r < hi; r += kWarps)
      for (int c = lane; c < p.rot; c += 32) cs[r * p.rot + c] = p.rope[(base + r) * p.rope_stride + c];
  }
  const int page = checked_page(p.batch, id, &g_kv_append_error);
  __syncthreads();
  if (page < 0) return;
  const int off = base % p.batch.page_size;

  // K and V: one head's block per warp
  for (int task = me; task < tasks; task += workers) {
    const int which = task >= p.n_kv_heads;
    const int h = which ? task - p.n_kv_heads : task;
    uint8_t* codes = p.pages[which] + int64_t(page) * p.page_stride +
                     (int64_t(h) * p.batch.page_size + off) * D + 8 * l;
    float* scale = p.scales[which] + int64_t(page) * p.scale_stride + h * (p.batch.page_size / kBlock) + off / kBlock;
    const float old = lo > 0 ? *scale : 0.0f;
    float x[PASSES][8];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) unpack8<T>(raw[i], x[i]);
    if (p.rope && !which) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = min(max(i * RPP + sub, lo), hi - 1);   // other rows hold zeros, which turn to zeros
        rotate8<LPR>(x[i], l, cs + r * p.rot, p.rot, p.interleaved);
      }
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[i][j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float sc = fmaxf(fmaxf(__fdiv_rn(top, Code<FMT>::kTop), old), kScaleFloor);
    const float inv = __fdiv_rn(1.0f, sc);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + sub;
      uint2* dst = reinterpret_cast<uint2*>(codes + r * D);
      if (r >= lo && r < hi) {
        *dst = quantize8<FMT>(x[i], sc, inv);
      } else if (r < lo && sc > old) {
        const uint2 c = *dst;
        float t[8];
        Code<FMT>::decode4(c.x, t);
        Code<FMT>::decode4(c.y, t + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = t[j] * old;
          t[j] = quotient_odd(y, fmaf(t[j], old, -y), sc, inv);
        }
        *dst = make_uint2(Code<FMT>::encode4(t), Code<FMT>::encode4(t + 4));
      }
    }
    __syncwarp();   // every lane has read the old scale
    if (lane == 0 && sc != old) *scale = sc;
    if (task + workers < tasks) fetch(task + workers);
  }

  // q: rows of (token, head), RPP rows per warp pass
  if (p.q) {
    const int rows = (hi - lo) * p.n_q_heads;
    constexpr int U = 4;
    // (the last warps first: with few tokens the first ones have a head's keys or values)
    for (int r0 = (workers - 1 - me) * RPP * U; r0 < rows; r0 += workers * RPP * U) {
      uint4 raw[U];
      int tok[U], head[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * RPP + sub;
        raw[u] = make_uint4(0, 0, 0, 0);
        tok[u] = r < rows ? lo + r / p.n_q_heads : -1;
        head[u] = r % p.n_q_heads;
        if (tok[u] >= 0)
          raw[u] = *reinterpret_cast<const uint4*>(p.q + int64_t(t0 + tok[u]) * p.q_stride + head[u] * D + 8 * l);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p.rope) {
          float x[8];
          unpack8<T>(raw[u], x);
          rotate8<LPR>(x, l, cs + max(tok[u], lo) * p.rot, p.rot, p.interleaved);
          raw[u] = pack8<T>(x);
        }
        if (tok[u] >= 0)
          *reinterpret_cast<uint4*>(p.q_out + int64_t(t0 + tok[u]) * p.q_out_stride + head[u] * D + 8 * l) = raw[u];
      }
    }
  }
}

struct DequantParams {
  Batch batch;
  const uint8_t* pages[2];
  const float* scales[2];
  int64_t page_stride, scale_stride;
  uint16_t* out[2];
  int32_t n_kv_heads;
};

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads) dequant_kv_kernel(const __grid_constant__ DequantParams p) {
  constexpr int LPR = D / 8;
  __shared__ int64_t scratch[40];
  pdl_launch();
  pdl_wait();
  int64_t rest;
  const int64_t slot = blockIdx.x;
  const int b = locate(
      p.batch.n_seqs, scratch, [&](int i) { return int64_t(touched(load_seq(p.batch, i, &g_kv_append_error))); },
      [&](int64_t) { return slot; }, &rest, static_cast<int64_t*>(nullptr));
  if (b < 0) return;
  const Seq s = load_seq(p.batch, b, &g_kv_append_error);
  const int p0 = max(s.past, 0);
  const int base = (p0 / kBlock + int(rest)) * kBlock;
  const int lo = max(base, p0) - base, hi = min(base + kBlock, s.len) - base;
  const int page = checked_page(
      p.batch, p.batch.table[int64_t(b) * p.batch.table_stride + base / p.batch.page_size], &g_kv_append_error);
  if (page < 0) return;
  const int t0 = s.t0 + (base - s.past);
  const int off = base % p.batch.page_size;
  const int per_row = p.n_kv_heads * LPR;
  const int items = 2 * (hi - lo) * per_row;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < items; i += gridDim.y * kThreads) {
    const int which = i >= items / 2;
    const int j = which ? i - items / 2 : i;
    const int r = lo + j / per_row, h = j % per_row / LPR, l = j % LPR;
    const uint2 c = *reinterpret_cast<const uint2*>(p.pages[which] + int64_t(page) * p.page_stride +
                                                    (int64_t(h) * p.batch.page_size + off + r) * D + 8 * l);
    const float sc = p.scales[which][int64_t(page) * p.scale_stride + h * (p.batch.page_size / kBlock) + off / kBlock];
    float t[8];
    Code<FMT>::decode4(c.x, t);
    Code<FMT>::decode4(c.y, t + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] *= sc;
    *reinterpret_cast<uint4*>(p.out[which] + (int64_t(t0 + r) * p.n_kv_heads + h) * D + 8 * l) = pack8<T>(t);
  }
}

// CTAs along y for `blocks` blocks of `work` warp tasks each: enough that a
// few tokens still use many SMs, no more than there are tasks.
int spread(int64_t blocks, int64_t tasks, int sms) {
  const int64_t want = (2 * sms + blocks - 1) / blocks, most = (tasks + kWarps - 1) / kWarps;
  return int(want < 1 ? 1 : want > most ? most : want);
}

template <typename P>
awq_status_t launch(void (*fn)(P), dim3 grid, const P& p, void* stream) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t lc = overlapped(grid, kThreads, 0, stream, &attr);
  if (cudaLaunchKernelEx(&lc, fn, p) != cudaSuccess) {
    cudaGetLastError();
    return AWQ_ERR_CUDA;
  }
  return AWQ_OK;
}

// The instantiation for (dtype, head_dim, format).
template <typename T>
void (*append_fn(int d, int fmt))(AppendParams) {
  if (d == 128) return fmt == AWQ_KV_INT8 ? append_kernel<T, 128, AWQ_KV_INT8> : append_kernel<T, 128, AWQ_KV_E4M3>;
  return fmt == AWQ_KV_INT8 ? append_kernel<T, 64, AWQ_KV_INT8> : append_kernel<T, 64, AWQ_KV_E4M3>;
}
template <typename T>
void (*dequant_fn(int d, int fmt))(DequantParams) {
  if (d == 128)
    return fmt == AWQ_KV_INT8 ? dequant_kv_kernel<T, 128, AWQ_KV_INT8> : dequant_kv_kernel<T, 128, AWQ_KV_E4M3>;
  return fmt == AWQ_KV_INT8 ? dequant_kv_kernel<T, 64, AWQ_KV_INT8> : dequant_kv_kernel<T, 64, AWQ_KV_E4M3>;
}

// Blocks that n_tokens rows of n_seqs sequences can touch: a run of n
// positions touches at most n, and at most (n + 30) / 16, of them.
int64_t slots(int64_t n_tokens, int64_t n_seqs) {
  const int64_t most = n_tokens / kBlock + 2 * n_seqs;
  return n_tokens < most ? n_tokens : most;
}

awq_status_t sm_count(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return AWQ_ERR_CUDA;
  }
  return AWQ_OK;
}

}  // namespace

awq_status_t append_take_error(uint32_t* word, cudaStream_t s) {
  const uint32_t zero = 0;
  if (cudaMemcpyFromSymbolAsync(word, g_kv_append_error, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_kv_append_error, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return AWQ_ERR_CUDA;
  return AWQ_OK;
}

}  // namespace kv
}  // namespace awq

extern "C" awq_status_t awq_kv_append(const awq_kv_cache_t* cache, const awq_kv_batch_t* batch, int64_t n_tokens,
                                      int32_t dtype, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                      int64_t v_stride, const uint16_t* q, int64_t q_stride, int32_t n_q_heads,
                                      const awq_kv_rope_t* rope, uint16_t* q_out, int64_t q_out_stride, void* stream) {
  using namespace awq;
  using namespace awq::kv;
  awq_status_t st;
  if ((st = check_cache(cache)) != AWQ_OK || (st = check_batch(batch, n_tokens)) != AWQ_OK ||
      (st = check_capacity(cache, batch)) != AWQ_OK)
    return st;
  if (!check_dtype(dtype)) return AWQ_ERR_UNSUPPORTED;
  if (rope) {
    if (rope->rot_dim < 16 || rope->rot_dim % 16 || rope->rot_dim > cache->head_dim) return AWQ_ERR_SHAPE;
    if (rope->n_positions < 0 || rope->n_positions > INT32_MAX || rope->row_stride < rope->rot_dim) return AWQ_ERR_SHAPE;
    if (rope->interleaved != 0 && rope->interleaved != 1) return AWQ_ERR_UNSUPPORTED;
  }
  if ((q != nullptr) != (q_out != nullptr)) return AWQ_ERR_NULL;
  if (q && (n_q_heads < 1 || n_q_heads > 65536)) return AWQ_ERR_SHAPE;
  if (n_tokens == 0 || batch->n_seqs == 0) return AWQ_OK;
  if ((st = check_pointers(cache, batch)) != AWQ_OK) return st;
  if ((st = check_rows(k, k_stride, cache->n_kv_heads, cache->head_dim)) != AWQ_OK ||
      (st = check_rows(v, v_stride, cache->n_kv_heads, cache->head_dim)) != AWQ_OK)
    return st;
  if (q && ((st = check_rows(q, q_stride, n_q_heads, cache->head_dim)) != AWQ_OK ||
            (st = check_rows(q_out, q_out_stride, n_q_heads, cache->head_dim)) != AWQ_OK))
    return st;
  if (rope && !rope->table) return AWQ_ERR_NULL;
  if (rope && (reinterpret_cast<uintptr_t>(rope->table) & 3u)) return AWQ_ERR_ALIGN;

  AppendParams p = {};
  p.batch = make_batch(cache, batch, n_tokens);
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  if (rope) {
    p.rope = rope->table;
    p.rope_stride = rope->row_stride;
    p.rope_rows = int32_t(rope->n_positions);
    p.rot = rope->rot_dim;
    p.interleaved = rope->interleaved;
  }
  p.pages[0] = cache->k_pages;
  p.pages[1] = cache->v_pages;
  p.scales[0] = cache->k_scales;
  p.scales[1] = cache->v_scales;
  p.page_stride = cache->page_stride;
  p.scale_stride = cache->scale_stride;
  p.n_q_heads = q ? n_q_heads : 0;
  p.n_kv_heads = cache->n_kv_heads;
  int sms = 0;
  if ((st = sm_count(&sms)) != AWQ_OK) return st;
  const int64_t blocks = slots(n_tokens, batch->n_seqs);
  // warp tasks of a block: a head's K or V, or a pass of q rows
  const int64_t per_pass = 4 * 32 / (cache->head_dim / 8);
  const int64_t rows = int64_t(p.n_q_heads) * (n_tokens < kBlock ? n_tokens : kBlock);
  const int y = spread(blocks, 2 * cache->n_kv_heads + (rows + per_pass - 1) / per_pass, sms);
  return launch(dtype == AWQ_KV_FP16 ? append_fn<__half>(cache->head_dim, cache->format)
                                     : append_fn<__nv_bfloat16>(cache->head_dim, cache->format),
                dim3(unsigned(blocks), unsigned(y)), p, stream);
}

extern "C" awq_status_t awq_kv_dequant(const awq_kv_cache_t* cache, const awq_kv_batch_t* batch, int64_t n_tokens,
                                       int32_t dtype, uint16_t* k_out, uint16_t* v_out, void* stream) {
  using namespace awq;
  using namespace awq::kv;
  awq_status_t st;
  if ((st = check_cache(cache)) != AWQ_OK || (st = check_batch(batch, n_tokens)) != AWQ_OK ||
      (st = check_capacity(cache, batch)) != AWQ_OK)
    return st;
  if (!check_dtype(dtype)) return AWQ_ERR_UNSUPPORTED;
  if (n_tokens == 0 || batch->n_seqs == 0) return AWQ_OK;
  if ((st = check_pointers(cache, batch)) != AWQ_OK) return st;
  const int64_t width = int64_t(cache->n_kv_heads) * cache->head_dim;
  if ((st = check_rows(k_out, width, cache->n_kv_heads, cache->head_dim)) != AWQ_OK ||
      (st = check_rows(v_out, width, cache->n_kv_heads, cache->head_dim)) != AWQ_OK)
    return st;
  DequantParams p = {};
  p.batch = make_batch(cache, batch, n_tokens);
  p.pages[0] = cache->k_pages;
  p.pages[1] = cache->v_pages;
  p.scales[0] = cache->k_scales;
  p.scales[1] = cache->v_scales;
  p.page_stride = cache->page_stride;
  p.scale_stride = cache->scale_stride;
  p.out[0] = k_out;
  p.out[1] = v_out;
  p.n_kv_heads = cache->n_kv_heads;
  int sms = 0;
  if ((st = sm_count(&sms)) != AWQ_OK) return st;
  const int64_t blocks = slots(n_tokens, batch->n_seqs);
  const int y = spread(blocks, (2 * kBlock * width / 8 + 31) / 32, sms);
  return launch(dtype == AWQ_KV_FP16 ? dequant_fn<__half>(cache->head_dim, cache->format)
                                     : dequant_fn<__nv_bfloat16>(cache->head_dim, cache->format),
                dim3(unsigned(blocks), unsigned(y)), p, stream);
}

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
// and scales are fp32. The quotients are exact: for int8 codes rounded as the
// real numbers they are, for e4m3 codes to fp32 and from there. 16-bit values
// over the block's largest fall on the border between two codes often enough
// (one in 10^4 or so) that a reciprocal's error would show in the cache
// (0.0006 against 0.0002 of an e4m3 cache's values, in the 2-norm), so a
// product that comes near a border is settled by a division.
//
// What bounds it: HBM bytes for prompts, launch and load latency for single
// tokens. Hence one CTA per touched block of 16 tokens (so that a scale and
// its codes have one writer and no atomics) with the heads spread over
// blockIdx.y when there are few blocks; the block's table rows are read once
// into shared memory and used for every head; two warps hold a head's whole
// block in registers (one read of K and V: the maximum and the codes come
// from the same values).
//
// Measured on one B200, on the GPU, 32 / 8 heads of 128, e4m3: 8319 prompt
// tokens 61 us (keys and values alone, not turned, 27), read back in 15; a
// token of one sequence 4, read back in 2. Heads of 128 spill (56 bytes for
// int8, 104 to 120 for e4m3, at 80 registers for three CTAs per SM).

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

// max(a, |x|, |y|), NaN if one of them is: a block with a NaN gets that as its scale and does not look sound.
__device__ __forceinline__ float max_abs_nan(float a, float x, float y) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(x), "f"(y));
  return r;
}

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x;
  v[1] = f.y;
  v[2] = f.z;
  v[3] = f.w;
}

// The rotation of channels 8l .. 8l+7 of a row (l: the lane's place among the
// row's lanes) by the angles of one position.
struct Turn {
  float c[8], s[8];   // interleaved: four of each
  int src;            // half-width pairs: the lane with the partner channels
  bool in, interleaved;

  // cs: the position's cosines and sines in shared memory.
  __device__ __forceinline__ void load(int l, const float* cs, int rot, bool inter) {
    const int half = rot >> 1, d0 = 8 * l, lane = threadIdx.x & 31;
    interleaved = inter;
    in = d0 < rot;
    src = lane;
    if (interleaved) {
      const float* at = cs + (in ? d0 >> 1 : 0);
      load4(at, c);
      load4(at + half, s);
      return;
    }
    const bool low = d0 < half;
    const float* at = cs + (in ? (low ? d0 : d0 - half) : 0);
    load4(at, c);
    load4(at + 4, c + 4);
    load4(at + half, s);
    load4(at + half + 4, s + 4);
    if (in) src = low ? lane + (half >> 3) : lane - (half >> 3);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = low ? -s[j] : s[j];
  }
  // (all lanes of the warp together)
  __device__ __forceinline__ void apply(float (&x)[8]) const {
    if (interleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = x[2 * j], b = x[2 * j + 1];
        if (in) {
          x[2 * j] = a * c[j] - b * s[j];
          x[2 * j + 1] = b * c[j] + a * s[j];
        }
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = __shfl_sync(0xffffffffu, x[j], src);
      if (in) x[j] = x[j] * c[j] + y * s[j];
    }
  }
};

// x / s (x = hi + lo), inv = 1 / s, ready to be rounded to a code. e4m3: to
// the nearest fp32. int8: rounded to odd in fp32 (cut off, with the last bit
// set where anything was cut), so that rounding it again rounds the quotient
// itself. The remainder fma(-q, s, hi) is exact.
template <int FMT>
__device__ __forceinline__ float quotient(float hi, float lo, float s, float inv) {
  float q = hi * inv;
  if (q == 0.0f) return q;   // keeps its sign
  q = fmaf(fmaf(-q, s, hi), inv, q);
  const float r = fmaf(-q, s, hi) + lo;
  if constexpr (FMT == AWQ_KV_E4M3) return fmaf(r, inv, q);
  uint32_t bits = __float_as_uint(q);
  if (r != 0.0f) bits = (bits - ((r < 0.0f) != (q < 0.0f) ? 1u : 0u)) | 1u;
  return __uint_as_float(bits);
}

// a b cut off to fp32 with the last bit set where anything was cut (rounded to
// odd), so that rounding it to 16 bits rounds the product itself.
__device__ __forceinline__ float product_to_odd(float a, float b) {
  const float p = __fmul_rz(a, b), r = fmaf(a, b, -p);   // r is exact; NaN beside an infinity, which stays
  return fabsf(r) > 0.0f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}

// The codes of eight values over the scale s (none above it by more than the
// rounding of top / R). Products by inv give the quotients within 3 ulp; if
// one of them comes that near to a border between two codes, all eight are
// divided.
template <int FMT>
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], float s, float inv) {
  if constexpr (FMT == AWQ_KV_INT8) {
    // x inv + 1.5 * 2^23 + 128 ends in the rounded integer, offset by 128; |x inv - integer| near 1/2 is a border
    constexpr float kMagic = 12583040.0f;
    float y[8], far = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = fmaf(x[j], inv, kMagic);
      far = fmaxf(far, fabsf(fmaf(x[j], inv, -(y[j] - kMagic))));
    }
    if (far > 0.4999f) {   // 127 * 3 * 2^-24 < 10^-4
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = rintf(quotient<FMT>(x[j], 0.0f, s, inv)) + kMagic;
    }
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t lo = __byte_perm(__float_as_uint(y[4 * k]), __float_as_uint(y[4 * k + 1]), 0x0040);
      const uint32_t hi = __byte_perm(__float_as_uint(y[4 * k + 2]), __float_as_uint(y[4 * k + 3]), 0x0040);
      w[k] = __byte_perm(lo, hi, 0x5410);
    }
    return make_uint2(w[0], w[1]);
  } else {
    // normal codes: the 20 bits that go are near their middle; subnormal ones (below 2^-6): always looked at
    float t[8];
    uint32_t near = 0xffffffffu, least = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      t[j] = x[j] * inv;
      const uint32_t b = __float_as_uint(t[j]);
      near = min(near, (b - 0x7fff8u) & 0xfffffu);
      least = min(least, (b & 0x7fffffffu) - 1u);
    }
    if (near <= 16u || least < 0x3c7fffffu) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = __fdiv_rn(x[j], s);
    }
    return make_uint2(Code<FMT>::encode4(t), Code<FMT>::encode4(t + 4));
  }
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 8;            // lanes per row of a head
  constexpr int RPP = 32 / LPR;         // rows per warp pass
  constexpr int PASSES = kBlock / 2 / RPP;   // a head's block is two warps' work, eight tokens each
  __shared__ int64_t scratch[40];
  __shared__ float tops[2][kWarps];
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
  const int teams = workers / 2, team = me / 2, r_first = (warp & 1) * (kBlock / 2) + sub;
  const int tasks = 2 * p.n_kv_heads;
  uint4 raw[PASSES];
  auto fetch = [&](int task) {                          // K or V rows of one head, zeros around the new ones
    const int which = task >= p.n_kv_heads;
    const int64_t stride = which ? p.v_stride : p.k_stride;
    const uint16_t* src = (which ? p.v : p.k) + int64_t(t0) * stride + (which ? task - p.n_kv_heads : task) * D + 8 * l;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = r_first + i * RPP;
      raw[i] = r >= lo && r < hi ? *reinterpret_cast<const uint4*>(src + r * stride) : make_uint4(0, 0, 0, 0);
    }
  };
  if (team < tasks) fetch(team);
  if (p.rope) {
    for (int r = lo + warp; r < hi; r += kWarps)
      for (int c = lane; c < p.rot; c += 32) cs[r * p.rot + c] = p.rope[(base + r) * p.rope_stride + c];
  }
  const int page = checked_page(p.batch, id, &g_kv_append_error);
  __syncthreads();
  if (page < 0) return;
  const int off = base % p.batch.page_size;

  // K and V
  for (int task = team, round = 0; task < tasks; task += teams, round ^= 1) {
    const int which = task >= p.n_kv_heads;
    const int h = which ? task - p.n_kv_heads : task;
    uint8_t* codes = p.pages[which] + int64_t(page) * p.page_stride +
                     (int64_t(h) * p.batch.page_size + off) * D + 8 * l;
    float* scale = p.scales[which] + int64_t(page) * p.scale_stride + h * (p.batch.page_size / kBlock) + off / kBlock;
    const float old = lo > 0 ? *scale : 0.0f;
    float x[PASSES][8];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      unpack8<T>(raw[i], x[i]);
      const int r = min(max(r_first + i * RPP, lo), hi - 1);   // other rows hold zeros, which turn to zeros
      if (p.rope && !which) {
        Turn turn;
        turn.load(l, cs + r * p.rot, p.rot, p.interleaved);
        turn.apply(x[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) top = max_abs_nan(top, x[i][j], x[i][j + 1]);
    }
    if (task + teams < tasks) fetch(task + teams);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_abs_nan(top, __shfl_xor_sync(0xffffffffu, top, o), 0.0f);
    if (lane == 0) tops[round][warp] = top;
    // (both warps have read the old scale, too)
    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
    top = max_abs_nan(top, tops[round][warp ^ 1], 0.0f);
    const float sc = max_abs_nan(__fdiv_rn(top, Code<FMT>::kTop), old, kScaleFloor);
    const float inv = __fdiv_rn(1.0f, sc);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = r_first + i * RPP;
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
          t[j] = quotient<FMT>(y, fmaf(t[j], old, -y), sc, inv);
        }
        *dst = make_uint2(Code<FMT>::encode4(t), Code<FMT>::encode4(t + 4));
      }
    }
    if (lane == 0 && !(warp & 1) && sc != old) *scale = sc;
  }

  // q: a warp takes U * RPP heads of a token, whose angles it loads once
  if (p.q) {
    constexpr int U = 4;
    const int per_token = (p.n_q_heads + U * RPP - 1) / (U * RPP);
    // (the last warps first: with few tokens the first ones have a head's keys or values)
    for (int u = workers - 1 - me; u < (hi - lo) * per_token; u += workers) {
      const int i = u / per_token, h0 = (u - i * per_token) * (U * RPP) + sub;
      const int64_t row = t0 + lo + i;
      const uint16_t* src = p.q + row * p.q_stride + 8 * l;
      uint16_t* dst = p.q_out + row * p.q_out_stride + 8 * l;
      uint4 raw[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int h = h0 + k * RPP;
        raw[k] = h < p.n_q_heads ? *reinterpret_cast<const uint4*>(src + h * D) : make_uint4(0, 0, 0, 0);
      }
      if (p.rope) {
        Turn turn;
        turn.load(l, cs + (lo + i) * p.rot, p.rot, p.interleaved);
#pragma unroll
        for (int k = 0; k < U; ++k) {
          float x[8];
          unpack8<T>(raw[k], x);
          turn.apply(x);
          raw[k] = pack8<T>(x);
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int h = h0 + k * RPP;
        if (h < p.n_q_heads) *reinterpret_cast<uint4*>(dst + h * D) = raw[k];
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
    for (int e = 0; e < 8; ++e) t[e] = product_to_odd(t[e], sc);
    *reinterpret_cast<uint4*>(p.out[which] + (int64_t(t0 + r) * p.n_kv_heads + h) * D + 8 * l) = pack8<T>(t);
  }
}

// CTAs along y for `blocks` blocks of `tasks` warp tasks each: one to two
// waves of CTAs, so that neither a few tokens nor a wave's remainder leave SMs idle,
// and no more than there are tasks.
int spread(int64_t blocks, int64_t tasks, int sms) {
  const int64_t want = (4 * sms + blocks - 1) / blocks, most = (tasks + kWarps - 1) / kWarps;
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
  // warp tasks of a block: two for a head's keys and two for its values, one for some heads of a token's q
  const int64_t heads = 4 * 32 / (cache->head_dim / 8), per_token = (p.n_q_heads + heads - 1) / heads;
  const int y = spread(blocks, 4 * cache->n_kv_heads + per_token * (n_tokens < kBlock ? n_tokens : kBlock), sms);
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

// Shared parts of the 8-bit paged KV cache's kernels: host-side checks, the
// batch's geometry on the device, and the 16-bit / 8-bit conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "awq_common.cuh"

namespace awq {
namespace kv {

constexpr int kBlock = AWQ_KV_BLOCK;          // tokens that share one scale
constexpr uint32_t kErrWait = 8u;             // awq_device_error bit 3
constexpr uint32_t kErrRange = 16u;           // awq_device_error bit 4
// Smallest scale. A block of zeros needs a scale above 0, because the
// attention adds log2 of the value scale to the logits; 2^-60 keeps its
// reciprocal (and sums of 2^60 over any context) inside fp32, and the weights
// of such a block inside it beside blocks of scales up to 2^40. fp16 values
// never reach it; bf16 values below 2^-61 become 0.
constexpr float kScaleFloor = 8.673617379884035e-19f;

// ---------------------------------------------------------------------------
// host-side checks
// ---------------------------------------------------------------------------
inline awq_status_t check_cache(const awq_kv_cache_t* c) {
  if (!c) return AWQ_ERR_NULL;
  if (c->format != AWQ_KV_INT8 && c->format != AWQ_KV_E4M3) return AWQ_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return AWQ_ERR_UNSUPPORTED;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->n_pages < 0 || c->n_pages > INT32_MAX) return AWQ_ERR_SHAPE;
  if (c->page_size < kBlock || c->page_size % kBlock || c->page_size > 65536) return AWQ_ERR_SHAPE;
  const int64_t page = int64_t(c->n_kv_heads) * c->page_size * c->head_dim;
  if (c->page_stride < page || c->page_stride % 16 || c->page_stride >= (int64_t(1) << 40)) return AWQ_ERR_SHAPE;
  if (c->scale_stride < int64_t(c->n_kv_heads) * (c->page_size / kBlock) || c->scale_stride >= (int64_t(1) << 40))
    return AWQ_ERR_SHAPE;
  return AWQ_OK;
}

// n_tokens: rows of q, k, v or of the outputs.
inline awq_status_t check_batch(const awq_kv_batch_t* b, int64_t n_tokens) {
  if (!b) return AWQ_ERR_NULL;
  if (b->n_seqs < 0 || b->n_seqs > (1 << 24) || b->max_pages < 0 || b->max_pages > (1 << 27)) return AWQ_ERR_SHAPE;
  if (b->table_stride < b->max_pages || b->max_q_len < 0) return AWQ_ERR_SHAPE;
  if (n_tokens < 0 || n_tokens > (int64_t(1) << 26)) return AWQ_ERR_SHAPE;
  return AWQ_OK;
}

// Positions are 32-bit integers: a sequence holds less than 2^31 tokens.
inline awq_status_t check_capacity(const awq_kv_cache_t* c, const awq_kv_batch_t* b) {
  return int64_t(b->max_pages) * c->page_size >= (int64_t(1) << 31) - 65536 ? AWQ_ERR_SHAPE : AWQ_OK;
}

// After the size checks, when there is work: the pointers.
inline awq_status_t check_pointers(const awq_kv_cache_t* c, const awq_kv_batch_t* b) {
  if (!b->block_table || !b->seq_lens || !b->q_indptr) return AWQ_ERR_NULL;
  if (!c->k_pages || !c->v_pages || !c->k_scales || !c->v_scales) return AWQ_ERR_NULL;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return AWQ_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(c->k_scales) | reinterpret_cast<uintptr_t>(c->v_scales) |
       reinterpret_cast<uintptr_t>(b->block_table) | reinterpret_cast<uintptr_t>(b->seq_lens) |
       reinterpret_cast<uintptr_t>(b->q_indptr)) & 3u)
    return AWQ_ERR_ALIGN;
  return AWQ_OK;
}

// Rows of heads x head_dim 16-bit values, `stride` values apart.
inline awq_status_t check_rows(const void* ptr, int64_t stride, int64_t heads, int64_t dim) {
  if (!ptr) return AWQ_ERR_NULL;
  if (stride < heads * dim || stride % 8 || stride >= (int64_t(1) << 40)) return AWQ_ERR_SHAPE;
  return aligned16(ptr) ? AWQ_OK : AWQ_ERR_ALIGN;
}

inline bool check_dtype(int32_t dtype) { return dtype == AWQ_KV_FP16 || dtype == AWQ_KV_BF16; }

// A launch that may start while the kernel before it on the stream finishes:
// the kernels wait (griddepcontrol.wait, in every thread) before they read or
// write anything that another kernel touches.
inline cudaLaunchConfig_t overlapped(dim3 grid, int threads, size_t smem, void* stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = static_cast<cudaStream_t>(stream);
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return lc;
}

// ---------------------------------------------------------------------------
// device side
// ---------------------------------------------------------------------------
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The batch as the kernels see it.
struct Batch {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* indptr;
  int64_t table_stride;
  int32_t n_seqs, n_tokens, max_pages, page_size;
  int64_t n_pages;
};

inline Batch make_batch(const awq_kv_cache_t* c, const awq_kv_batch_t* b, int64_t n_tokens) {
  Batch r;
  r.table = b->block_table;
  r.lens = b->seq_lens;
  r.indptr = b->q_indptr;
  r.table_stride = b->table_stride;
  r.n_seqs = b->n_seqs;
  r.n_tokens = int32_t(n_tokens);
  r.max_pages = b->max_pages;
  r.page_size = c->page_size;
  r.n_pages = c->n_pages;
  return r;
}

// a / b for a >= 0, b > 0: 64-bit division takes several hundred cycles, and
// both are nearly always short.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return (uint64_t(a | b) >> 32) ? a / b : int64_t(uint32_t(a) / uint32_t(b));
}

// One sequence: its tokens of this call are rows t0 .. t0 + n - 1, at
// positions past .. len - 1 (past is negative when the sequence is shorter
// than its rows: those rows have no position). The values come from device
// memory, so they are brought into range here, whatever they hold.
struct Seq {
  int t0, n, len, past;
};

__device__ __forceinline__ Seq load_seq(const Batch& a, int b, uint32_t* err) {
  Seq s;
  const int i0 = a.indptr[b], i1 = a.indptr[b + 1], raw = a.lens[b];
  s.t0 = min(max(i0, 0), a.n_tokens);
  s.n = min(max(i1, s.t0), a.n_tokens) - s.t0;
  s.len = min(max(raw, 0), a.max_pages * a.page_size);
  s.past = s.len - s.n;
  if (i0 < 0 || i1 < i0 || i1 > a.n_tokens || raw < 0 || raw > a.max_pages * a.page_size) atomicOr(err, kErrRange);
  return s;
}

// The page that holds position pos of sequence b, or -1 (recorded) where the
// table names none of the cache's.
__device__ __forceinline__ int checked_page(const Batch& a, int id, uint32_t* err) {
  if (id >= 0 && id < a.n_pages) return id;
  atomicOr(err, kErrRange);
  return -1;
}

// Finds the sequence that holds unit `target(total)` when sequence b has
// count(b) units. Every thread of the block calls it; `scratch` is shared
// memory of at least 40 int64. Each thread takes a run of sequences, the
// block scans the sums, and the thread whose run holds the target walks it.
// Returns the sequence (-1 when the target is at or past the total); *rest is
// the target's place in it.
template <class Count, class Target>
__device__ __forceinline__ int locate(int n_seqs, int64_t* scratch, Count count, Target target, int64_t* rest,
                                      int64_t* total_out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (n_seqs == 1) {   // nothing to search: one load's latency instead of a scan
    const int64_t only = count(0), goal = target(only);
    *rest = goal;
    if (total_out) *total_out = only;
    return goal < only ? 0 : -1;
  }
  const int run = (n_seqs + blockDim.x - 1) / blockDim.x;
  const int b0 = min(int(threadIdx.x) * run, n_seqs), b1 = min(b0 + run, n_seqs);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += count(b);
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  if (threadIdx.x == 0) scratch[33] = -1;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  const int64_t goal = target(total);
  int64_t at = before + inc - sum;
  if (goal >= at && goal < at + sum) {
    for (int b = b0; b < b1; ++b) {
      const int64_t c = count(b);
      if (goal < at + c) {
        scratch[33] = b;
        scratch[34] = goal - at;
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  *rest = scratch[34];
  if (total_out) *total_out = total;
  return int(scratch[33]);
}

template <typename T>
struct Half16;
template <>
struct Half16<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Half16<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Half16<T>::unpack(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Half16<T>::pack(x[0], x[1]), Half16<T>::pack(x[2], x[3]), Half16<T>::pack(x[4], x[5]),
                    Half16<T>::pack(x[6], x[7]));
}

// The 8-bit forms: int8 codes -127 .. 127 are held offset by 128, e4m3 codes
// as they are. encode4 takes values already divided by the scale.
template <int FMT>
struct Code;
template <>
struct Code<AWQ_KV_INT8> {
  static constexpr float kTop = 127.0f;
  static __device__ __forceinline__ uint32_t encode4(const float* t) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w |= uint32_t(int(fminf(fmaxf(rintf(t[i]), -127.0f), 127.0f)) + 128) << (8 * i);
    return w;
  }
  static __device__ __forceinline__ void decode4(uint32_t w, float* t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = float(int((w >> (8 * i)) & 0xffu) - 128);
  }
};
template <>
struct Code<AWQ_KV_E4M3> {
  static constexpr float kTop = 448.0f;
  static __device__ __forceinline__ uint32_t encode4(const float* t) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(t[0], t[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(t[2], t[3]), __NV_SATFINITE, __NV_E4M3);
    return a | (b << 16);
  }
  static __device__ __forceinline__ void decode4(uint32_t w, float* t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t((w >> (16 * i)) & 0xffffu), __NV_E4M3);
      const float2 f = __half22float2(__half2(r));
      t[2 * i] = f.x;
      t[2 * i + 1] = f.y;
    }
  }
};

}  // namespace kv
}  // namespace awq

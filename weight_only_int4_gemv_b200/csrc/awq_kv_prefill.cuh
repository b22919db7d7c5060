// The many-row kernel of awq_kv_attention (prompts, chunks of prompts),
// included by awq_kv_attention.cu inside namespace awq::kv.
//
// Mathematics: as for few rows (t = scale log2(e) s_k S + log2(s_v), p = 2^(t
// - m + 7), y = sum p c_v / sum (p / s_v)), over tiles of 128 rows by 128 keys.
//
// What bounds it: two products of 128 x 128 x head_dim and 128 x 128
// exponentials per tile, about equal at the tensor and the special-function
// units' rates; so both products run on tcgen05 and everything else is kept
// off the warps that do the softmax. One CTA per SM takes two row tiles (256
// rows of one key / value head: the rows of 256 / group tokens) against the
// same keys, so a code is turned into its fp16 form once for two products,
// and the softmax of one row tile runs while the other's products do.
//
// Warps:
//   0-15      softmax: a thread has half a row (64 of a tile's keys) of row
//             tile 0 (warps 0-3, 8-11) or 1 (4-7, 12-15); the halves exchange
//             their largest logits through shared memory. S comes from tensor
//             memory, the weights go back over it as fp16 (the A operand of
//             the second product). m is only raised when a logit passes it by
//             more than 8 (log2 units), so the outputs in tensor memory are
//             almost never rescaled.
//   16-19     codes to fp16 (exact) in the tensor core's 128-byte-swizzled
//             layout: keys K-major, values as they lie (MN-major); the
//             blocks' constants.
//   20        pages, scales and the tiles' descriptions, TMA of the codes.
//   21        the products: S0 = Q0 K^T, S1 = Q1 K^T, O0 += P0 V, O1 += P1 V.
//   22, 23    q rows to fp16, a segment ahead.
// Tensor memory: S0, S1 (128 columns each; a half row's P lies over its S), O0, O1.
//
// Work is laid end to end in units of 128 keys and cut evenly over the CTAs,
// as for few rows; split items meet in join_rows_kernel.
//
// Measured on one B200: chunks of up to 509 rows x 8 heads over up to 6001
// tokens, 8 key / value heads of 128, e4m3: 225 us, 679 TFLOP/s (40 % of a
// dense bf16 product's measured rate); a prompt of 2048, 32 / 8 heads, int8: 70
// us, 490 TFLOP/s; 4096 with a window of 1024: 126 us, 478. Two thirds of the
// tensor pipe's cycles are idle: a tile's softmax takes 2800 to 3900 cycles,
// its products 2000 and its exponentials alone about 1000. What stands between
// is exposed latency: S is read in steps of 32 columns, each waited for, once
// for the maximum and again for the weights; the halves of all rows of a row
// tile meet in between; the second product starts when all of P is there. The
// exponential unit is not the bound: every fourth (third, second) pair of
// exponentials as a polynomial on the FMA pipe took 71 (71, 74) us for the
// prompt.

constexpr int kTile = 128;                     // keys of a tile, and rows of a row tile
constexpr int kPairRows = 2 * kTile;
constexpr int kSoftmaxWarps = 16, kWidenWarps = 4;
constexpr int kPreThreads = (kSoftmaxWarps + kWidenWarps + 4) * 32;
// What a segment costs beyond its tiles (q rows, first S, epilogue), in tiles: the schedule counts every item as
// that much longer (1, 2, 3, 4: chunks of 509 rows over 6000 295, 254, 226, 226 us; a prompt of 2048 81, 72, 72, 73).
constexpr int kSegmentCost = 3;
constexpr float kLeastA = 7.888609052210118e-31f;    // 2^-100
constexpr float kSpoilt = 3.4028234663852886e38f;    // the largest number: no logit's size
constexpr int kRawSlots = 3, kHalfSlots = 3, kMetaSlots = 4;

enum : int {                                   // PreMeta::flags
  kAct0 = 1, kAct1 = 2,                        // the row tile sees some of these keys
  kBegin = 4, kEnd = 8,                        // first / last tile of the segment
  kBegin0 = 16, kBegin1 = 32,                  // the row tile's first tile of the segment
  kEnd0 = 64, kEnd1 = 128,                     // its last
  kHas0 = 256, kHas1 = 512,                    // the row tile has a tile in the segment
  kStop = 1024,                                // no more tiles
  kHoles = 2048                                // a block's page id is out of range
};

// 1 / l; 0 for a row that sees nothing, NaN for one that sees a spoilt block.
__device__ __forceinline__ float inverse(float m, float l) {
  return m == -INFINITY ? 0.0f : m >= kSpoilt ? __uint_as_float(0x7fffffffu) : __fdiv_rn(1.0f, l);
}

struct alignas(16) PreMeta {     // (its arrays are read two floats at a time)
  int pos, flags;
  int t0, row0, rows, past, head, dest;
  float ks[8], vs[8];            // the blocks' scales
  float a[8], lv[8], iv[8];      // scale log2(e) s_k, log2(s_v), 1 / s_v
  uint32_t missing;              // with kHoles: bit i: block i has no page
};

template <int D>
struct PreShared {
  uint8_t q[2][kTile * D * 2];
  uint8_t half[kHalfSlots][kTile * D * 2];
  uint8_t raw[kRawSlots][kTile * D];
  float factor[kMetaSlots][2][kTile];          // [segment][row tile][row]: a ring of as many segments as tiles
  float peak[2][2][2][kTile];                  // [tile parity][row tile][half][row]: a half row's largest logit
  float mass[2][2][kTile];                     // its sum of weights, at a segment's end
  PreMeta meta[kMetaSlots];
  uint64_t both[2];                            // the halves' exchange
  uint64_t meta_full[kMetaSlots], meta_empty[kMetaSlots];
  uint64_t raw_full[kRawSlots], raw_empty[kRawSlots];
  uint64_t half_full[kHalfSlots], half_empty[kHalfSlots];
  uint64_t q_full[2], q_free[2], s_full[2], p_ready[2], o_full[2], o_free[2], done;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// D += A B, both operands in shared memory
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(accumulate)
      : "memory");
}
// D += A B, A in tensor memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(accumulate)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// this warp's 32 lanes x 32 columns. The wait is in the same statement: nothing may read r before it.
__device__ __forceinline__ void tc_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}"
      ", [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), 
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tc_ld32(uint32_t a, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a)
      : "memory");
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 32 bytes to a 32-byte-aligned address
__device__ __forceinline__ void st_global_32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptors, 128-byte swizzle. K-major: 8-row groups
// 1024 bytes apart. MN-major (values: rows are keys, 64 channels a panel):
// panels kTile rows apart, 8-key groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t a) {
  return uint64_t((a >> 4) & 0x3FFF) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t a) {
  return uint64_t((a >> 4) & 0x3FFF) | (uint64_t(kTile * 128 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// One row pair: rows row0 .. of a sequence, the tiles each half sees, and
// their union (sink tiles, then tiles from w0).
struct Pair {
  int hi[2], lo[2];      // last (-1: none) and first window tile of each half
  int sink_tiles, w0, tiles;
};

__device__ __forceinline__ Pair pair_of(const AttentionParams& p, const Seq& s, int row0) {
  Pair r;
  const int rows = s.n * p.group;
  int hi = -1, lo = 1 << 30, low = 0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    r.hi[x] = -1;
    r.lo[x] = 0;
    const int first = row0 + x * kTile;
    if (first < rows) {
      const int p_low = s.past + first / p.group, p_high = s.past + (min(first + kTile, rows) - 1) / p.group;
      if (p_high >= 0) {
        r.hi[x] = p_high / kTile;
        const int start = window_start(p_low, p.window);
        r.lo[x] = start / kTile;
        if (x == 0 || hi < 0) low = start;
        hi = max(hi, r.hi[x]);
        lo = min(lo, r.lo[x]);
      }
    }
  }
  if (hi < 0) {          // rows that see nothing: one tile without keys, for their zeros
    r.sink_tiles = r.w0 = 0;
    r.tiles = 1;
    return r;
  }
  r.w0 = lo;
  r.sink_tiles = p.window ? min((min(p.sinks, low) + kTile - 1) / kTile, lo) : 0;
  r.tiles = r.sink_tiles + hi - lo + 1;
  return r;
}

// Units of 32 sequences, one to a lane: a lane counts a short one by itself, the warp the long ones in turn. (133
// sequences of up to 96 rows over 278 tokens, all in turn and like this: 125 and 31 us; 600 of up to 96 over 42: 484
// and 52.)
__device__ __forceinline__ int64_t units_of(const AttentionParams& p, const Seq& mine, int lane) {
  constexpr int kShort = 8;
  const int all = (mine.n * p.group + kPairRows - 1) / kPairRows;
  unsigned left = __ballot_sync(0xffffffffu, all > kShort);
  Seq s = mine;
  int first = 0, step = 1, pairs = all > kShort ? 0 : all;
  int64_t units = 0;
#pragma unroll 1
  for (int who = lane;;) {
    int64_t sum = 0;
#pragma unroll 1
    for (int i = first; i < pairs; i += step) sum += pair_of(p, s, i * kPairRows).tiles + kSegmentCost;
    if (step > 1) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (who == lane) units += sum;
    if (!left) break;
    who = __ffs(left) - 1;
    left &= left - 1;
    first = lane;
    step = 32;
    s = {__shfl_sync(0xffffffffu, mine.t0, who), __shfl_sync(0xffffffffu, mine.n, who),
         __shfl_sync(0xffffffffu, mine.len, who), __shfl_sync(0xffffffffu, mine.past, who)};
    pairs = __shfl_sync(0xffffffffu, all, who);
  }
  return units * p.n_kv_heads;
}

// 16 raw codes to 16 fp16 numbers, two 16-byte chunks.
template <int FMT>
__device__ __forceinline__ void widen16(const uint4& c, uint4& a, uint4& b) {
  a = make_uint4(code_pair<FMT, 0>(c.x), code_pair<FMT, 2>(c.x), code_pair<FMT, 0>(c.y), code_pair<FMT, 2>(c.y));
  b = make_uint4(code_pair<FMT, 0>(c.z), code_pair<FMT, 2>(c.z), code_pair<FMT, 0>(c.w), code_pair<FMT, 2>(c.w));
}

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Largest (smallest) of 16.
template <class Op3>
__device__ __forceinline__ float extreme16(const uint32_t* r, Op3 op) {
  auto f = [&](int i) { return __uint_as_float(r[i]); };
  const float a = op(f(0), f(1), f(2)), b = op(f(3), f(4), f(5)), c = op(f(6), f(7), f(8)), d = op(f(9), f(10), f(11));
  return op(op(a, b, f(12)), op(c, d, f(13)), op(f(14), f(15), f(15)));
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kPreThreads, 1)
prefill_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ AttentionParams p) {
  using Sh = PreShared<D>;
  constexpr uint32_t kIdescS = (1u << 4) | (uint32_t(kTile >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
  constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
  extern __shared__ uint8_t smem_raw[];
  // (an offset from the array, not a rounded address: the compiler then knows it is shared memory)
  Sh& sh = *reinterpret_cast<Sh*>(smem_raw + ((0u - smem_u32(smem_raw)) & 1023u));
  // The warps' parts by number (a scheduler has every fourth warp): 16, 18, 19, 20 widen, so that the products' warp,
  // 17, shares its scheduler with no widening one; 21 and 23 bring q, 22 the schedule.
  const int lane = threadIdx.x & 31, hw_warp = threadIdx.x >> 5;
  const int warp = hw_warp < 17 ? hw_warp : hw_warp == 17 ? 21 : hw_warp < 21 ? hw_warp - 1 : hw_warp == 21 ? 22 : hw_warp == 22 ? 20 : 23;
  volatile int* abort = &sh.abort;
  uint32_t* err = &g_kv_attention_error;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMetaSlots; ++i) {
      mbar_init(&sh.meta_full[i], 33);
      mbar_init(&sh.meta_empty[i], kSoftmaxWarps + kWidenWarps + 3);   // all warps but the one that writes it
    }
    for (int i = 0; i < kRawSlots; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], 4);
    }
    for (int i = 0; i < kHalfSlots; ++i) {
      mbar_init(&sh.half_full[i], 4);
      mbar_init(&sh.half_empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh.q_full[x], 2);
      mbar_init(&sh.q_free[x], 1);
      mbar_init(&sh.s_full[x], 1);
      mbar_init(&sh.p_ready[x], kSoftmaxWarps / 2);
      mbar_init(&sh.both[x], kSoftmaxWarps / 2);
      mbar_init(&sh.o_full[x], 1);
      mbar_init(&sh.o_free[x], kSoftmaxWarps / 2);
    }
    mbar_init(&sh.done, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == kSoftmaxWarps + kWidenWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  pdl_launch();
  pdl_wait();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem;
  // one answer for the whole warp, so that its collective instructions stay together when a wait gives up
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_small(bar, parity, p.wait, abort, err)) != 0;
  };

  if (warp < kSoftmaxWarps) {
    // -------------------------------------------------------------- softmax
    const int x = (warp >> 2) & 1, half = warp >> 3, row = threadIdx.x & (kTile - 1);
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    // this half's columns of S (its weights lie over the first of them) and of O
    const uint32_t ts = tmem + lanes + x * kTile + half * (kTile / 2);
    const uint32_t to = tmem + lanes + 2 * kTile + x * D + half * (D / 2);
    float m = -INFINITY, l = 0.0f, factor = 1.0f;      // l: of this half
    int pv = 0, p_row = 0, p_low = 0, p_high = 0;      // pv: products into O in this segment
    uint32_t s_ph = 0, o_ph = 0, both_ph = 0;          // parity of the next S, of the next O, of the next exchange
    uint32_t seg = 0;
    for (int it = 0;; ++it) {
      const int mi = it % kMetaSlots;
      if (!wait(&sh.meta_full[mi], (it / kMetaSlots) & 1)) break;
      const PreMeta& me = sh.meta[mi];
      const int flags = me.flags;
      if (flags & kStop) break;
      if (flags & kBegin) {
        m = -INFINITY;
        l = 0.0f;
        pv = 0;
        const int r0 = me.row0 + x * kTile, r1 = min(r0 + kTile, me.row0 + me.rows) - 1;
        p_low = me.past + r0 / p.group;
        p_high = me.past + r1 / p.group;
        p_row = me.past + (r0 + row) / p.group;
      }
      if (flags & (x ? kAct1 : kAct0)) {
        const int pos = me.pos;
        const bool all = !(flags & kHoles) && pos + kTile - 1 <= p_low &&
                         (p.window == 0 || pos > p_high - p.window || pos + kTile <= p.sinks);
        const int k0 = half * (kTile / 2);             // the first key's column
        const int hi = p_row - pos - k0, lo = p.window ? hi - p.window + 1 : 0,
                  sk = p.window ? p.sinks - pos - k0 : 0;
        if (!wait(&sh.s_full[x], s_ph)) break;
        s_ph ^= 1;
        tc_after();
        // (written before the row tile's first S was computed)
        if (std::is_same<T, __nv_bfloat16>::value && pv == 0) factor = sh.factor[seg % kMetaSlots][x][row];
        const bool flip = p.scale_log2 < 0.0f;
        // t = a S + log2(s_v); |a| stays above 0, so that an infinite S is an infinite t (2^-100 S is no logit)
        auto block_a = [&](float a) {
          if constexpr (std::is_same<T, __nv_bfloat16>::value) a = copysignf(fmaxf(fabsf(a * factor), kLeastA), a);
          return a;
        };
        if (!all) {
          // masked columns of S become the infinity that a's sign takes to -inf
#pragma unroll 1
          for (int c = 0; c < kTile / 64; ++c) {
            uint32_t vis = low_bits(hi - 32 * c + 1) & (~low_bits(lo - 32 * c) | low_bits(sk - 32 * c));
            if (flags & kHoles) {      // the keys of a missing block are whatever shared memory held
              const uint32_t gone = me.missing >> (half * 4 + 2 * c);
              vis &= ~((gone & 1u) * 0xffffu | ((gone >> 1) & 1u) * 0xffff0000u);
            }
            if (__all_sync(0xffffffffu, vis == 0xffffffffu)) continue;
            uint32_t r[32];
            tc_ld32(ts + c * 32, r);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(vis & (1u << k))) r[k] = flip ? 0x7f800000u : 0xff800000u;
            tc_st32(ts + c * 32, r);
          }
          tc_wait_st();
        }
        // Two passes over S, each a short rolled loop: straight code for a whole tile lives on instruction cache
        // misses. The largest logit: per block the extreme of S, then its t.
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kTile / 64; ++c) {
          uint32_t r[32];
          const int b = half * 4 + 2 * c;
          const float2 a = *reinterpret_cast<const float2*>(&me.a[b]), lv = *reinterpret_cast<const float2*>(&me.lv[b]);
          tc_ld32(ts + c * 32, r);
          float e0, e1;
          if (flip) {
            e0 = extreme16(r, min3);
            e1 = extreme16(r + 16, min3);
          } else {
            e0 = extreme16(r, max3);
            e1 = extreme16(r + 16, max3);
          }
          top = max3(top, fmaf(e0, block_a(a.x), lv.x), fmaf(e1, block_a(a.y), lv.y));
        }
        // (the other half of the row has its own part of S and the same m)
        float* peak = &sh.peak[o_ph][x][0][row];
        peak[half * kTile] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.both[x]);
        if (!wait(&sh.both[x], both_ph)) break;
        both_ph ^= 1;
        top = fmaxf(top, peak[(half ^ 1) * kTile]);
        if (__any_sync(0xffffffffu, top > m + kSlack)) {
          const float raised = fmaxf(m, top);
          const float f = raised == -INFINITY ? 1.0f : exp2_fast(m - raised);
          if (pv > 0) {
            // the products so far are in, and are brought to the new maximum
            if (!wait(&sh.o_full[x], o_ph ^ 1)) break;
            tc_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t y[16];
              tc_ld16(to + c * 16, y);
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
              tc_st16(to + c * 16, y);
            }
          }
          l *= f;
          m = raised;
        }
        // The weights, over the S columns.
        const float base = m == -INFINITY ? 0.0f : m - kLift;
#pragma unroll 1
        for (int c = 0; c < kTile / 64; ++c) {
          uint32_t r[32], pk[16];
          const int b = half * 4 + 2 * c;
          const float2 a2 = *reinterpret_cast<const float2*>(&me.a[b]), lv = *reinterpret_cast<const float2*>(&me.lv[b]),
                       iv = *reinterpret_cast<const float2*>(&me.iv[b]);
          const float a[2] = {block_a(a2.x), block_a(a2.y)}, d[2] = {lv.x - base, lv.y - base}, is[2] = {iv.x, iv.y};
          tc_ld32(ts + c * 32, r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 16 * h; e < 16 * h + 16; e += 2) {
              const float2 t = fma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])),
                                    make_float2(a[h], a[h]), make_float2(d[h], d[h]));
              const float2 w = make_float2(exp2_fast(t.x), exp2_fast(t.y));
              part = add2(part, w);
              pk[e / 2] = Half16<__half>::pack(w.x, w.y);
            }
            l = fmaf(part.x + part.y, is[h], l);
          }
          tc_st16(ts + c * 16, pk);
        }
        tc_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[x]);
        ++pv;
        o_ph ^= 1;
      }
      if (flags & kEnd) {
        const int r0 = x * kTile + row;
        const bool mine = r0 < me.rows;
        const int gr = me.row0 + r0, dest = me.dest;
        uint16_t* dst = p.out + int64_t(me.t0 + gr / p.group) * p.out_stride +
                        int64_t(me.head * p.group + gr % p.group) * D + half * (D / 2);
        const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
        float* part = p.part + int64_t(dest) * (kPairRows * (D + 2));
        if (pv > 0) {
          if (!wait(&sh.o_full[x], o_ph ^ 1)) break;
          tc_after();
          sh.mass[x][half][row] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.both[x]);
          if (!wait(&sh.both[x], both_ph)) break;
          both_ph ^= 1;
          l += sh.mass[x][half ^ 1][row];
        }
        const float inv = inverse(m, l);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t r[32];
          if (pv > 0) {
            tc_ld32(to + c * 32, r);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0;
          }
          if (mine && dest < 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              float v[8], w[8];
#pragma unroll
              for (int f = 0; f < 8; ++f) {
                v[f] = __uint_as_float(r[e + f]) * inv;
                w[f] = __uint_as_float(r[e + 8 + f]) * inv;
              }
              const uint4 a = pack8<T>(v), b = pack8<T>(w);
              if (wide) {
                st_global_32(dst + c * 32 + e, a, b);
              } else {
                *reinterpret_cast<uint4*>(dst + c * 32 + e) = a;
                *reinterpret_cast<uint4*>(dst + c * 32 + e + 8) = b;
              }
            }
          } else if (mine) {
            // four channels of a row together, rows side by side: the lanes' stores are contiguous
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + ((half * (D / 8) + c * 8 + e / 4) * kPairRows + r0) * 4) =
                  make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
          }
        }
        if (mine && dest >= 0 && half == 0) *reinterpret_cast<float2*>(part + kPairRows * D + 2 * r0) = make_float2(m, l);
        if (pv > 0) {
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.o_free[x]);
        }
        ++seg;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.meta_empty[mi]);
    }
  } else if (warp < kSoftmaxWarps + kWidenWarps) {
    // ---------------------------------------------------------- codes to fp16
    // A thread takes 16-byte chunk k of the rows r0, r0 + kRowStep, ...: 16 channels, chunks 2k and 2k + 1 (mod 8) of
    // its panel's row. Eight lanes read eight chunks at once, and write to eight different ones: with two panels,
    // lanes 4-7 take the row beside lanes 0-3's, whose chunks the swizzle puts on the other places.
    const int tid = (warp - kSoftmaxWarps) * 32 + lane;
    constexpr int CPR = D / 16, kRowStep = 128 / CPR;
    const int k = tid % CPR, r0 = D == 128 ? (tid >> 3) ^ (k >> 2) : tid / CPR;
    const int raw_at = r0 * D + k * 16, half_at = (k >> 2) * (kTile * 128) + r0 * 128;
    const int c0 = ((2 * (k & 3)) ^ (r0 & 7)) << 4, c1 = ((2 * (k & 3) + 1) ^ (r0 & 7)) << 4;
    int n = 0;                                  // tiles of codes converted
    for (int it = 0;; ++it) {
      const int mi = it % kMetaSlots;
      if (!wait(&sh.meta_full[mi], (it / kMetaSlots) & 1)) break;
      const PreMeta& me = sh.meta[mi];
      const int flags = me.flags;
      if (flags & kStop) break;
      const unsigned zeros = __ballot_sync(0xffffffffu, lane < 8 && me.vs[lane & 7] < kScaleFloor);
      if (tid < 8) {                             // (published with the keys)
        PreMeta& out = sh.meta[mi];
        // A scale that is no finite number of at least 0 must not reach the rows that do not see its block (there t is -inf by S, whatever
        // finite numbers stand here) and has to show in the others: their m becomes kSpoilt, which ends as NaN.
        const float ks = me.ks[tid], vs = me.vs[tid];
        const bool fine = ks >= 0.0f && vs >= 0.0f && ks + vs < INFINITY;
        const float a = fine ? fmaxf(fabsf(p.scale_log2) * kShift<FMT> * ks, kLeastA) : kLeastA;
        out.a[tid] = p.scale_log2 < 0.0f ? -a : a;
        // (a scale of 0, or below the smallest, counts as that here, which gives its keys their mass; its codes are made
        // 0 below)
        const float v = fmaxf(vs, kScaleFloor);
        out.lv[tid] = fine ? __log2f(v) : kSpoilt;
        out.iv[tid] = fine ? __fdividef(1.0f / kShift<FMT>, v) : 1.0f;   // (O holds codes / kShift)
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.meta_empty[mi]);
      if (!(flags & (kAct0 | kAct1))) continue;  // a tile without keys
      bool ok = true;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++n) {
        const int rs = n % kRawSlots, hs = n % kHalfSlots;
        if (!wait(&sh.raw_full[rs], (n / kRawSlots) & 1) || !wait(&sh.half_empty[hs], ((n / kHalfSlots) & 1) ^ 1)) {
          ok = false;
          break;
        }
        const uint8_t* raw = sh.raw[rs] + raw_at;
        uint8_t* half = sh.half[hs] + half_at;
#pragma unroll 4
        for (int i = 0; i < kTile / kRowStep; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(raw + i * kRowStep * D);
          uint4 a, b;
          widen16<FMT>(w, a, b);
          *reinterpret_cast<uint4*>(half + i * kRowStep * 128 + c0) = a;
          *reinterpret_cast<uint4*>(half + i * kRowStep * 128 + c1) = b;
        }
        if (kv && zeros) {                        // values of scale 0, whatever their codes
#pragma unroll 1
          for (int i = 0; i < kTile / kRowStep; ++i)
            if ((zeros >> ((r0 + i * kRowStep) / kBlock)) & 1u)
              *reinterpret_cast<uint4*>(half + i * kRowStep * 128 + c0) =
                  *reinterpret_cast<uint4*>(half + i * kRowStep * 128 + c1) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.half_full[hs]);
          mbar_arrive(&sh.raw_empty[rs]);
        }
      }
      if (!ok) break;
    }
  } else if (warp == kSoftmaxWarps + kWidenWarps) {
    // --------------------------------------------- the schedule, pages, copies
    const Batch& a = p.batch;
    Join join;
    join.last = -1;
    int it = 0, n = 0;
    bool ok = true;
    // The first walk over the sequences counts the units, the second one hands out this CTA's.
    int64_t total = 0, per = 0, u0 = 0, u1 = 0;
    int64_t u = 0;                               // units before the sequence
    bool counting = true;
#pragma unroll 1
    for (int b0 = 0; ok; b0 += 32) {
      if (b0 >= a.n_seqs) {
        if (!counting) break;
        counting = false;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        per = divide(total + gridDim.x - 1, gridDim.x);
        u0 = per * blockIdx.x;
        u1 = min(u0 + per, total);
        b0 = -32;
        continue;
      }
      if (!counting && u >= u1) break;
      Seq mine = {0, 0, 0, 0};
      if (b0 + lane < a.n_seqs) mine = load_seq(a, b0 + lane, err);
      const int64_t own_units = units_of(p, mine, lane);
      if (counting) {
        total += own_units;
        continue;
      }
      int64_t before = own_units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      const unsigned reach = __ballot_sync(0xffffffffu, u + before > u0);
      if (!reach) {
        u += __shfl_sync(0xffffffffu, before, 31);
        continue;
      }
      const int i0 = __ffs(reach) - 1;           // the first sequence with units of this run
      u += __shfl_sync(0xffffffffu, before - own_units, i0);
      for (int i = i0; i < min(32, a.n_seqs - b0) && u < u1 && ok; ++i) {
        const Seq s = {__shfl_sync(0xffffffffu, mine.t0, i), __shfl_sync(0xffffffffu, mine.n, i),
                       __shfl_sync(0xffffffffu, mine.len, i), __shfl_sync(0xffffffffu, mine.past, i)};
        const int64_t units = __shfl_sync(0xffffffffu, own_units, i);
        const int32_t* table = a.table + int64_t(b0 + i) * a.table_stride;
        const int rows = s.n * p.group, pairs = (rows + kPairRows - 1) / kPairRows;
        int64_t begin = u;                       // units before the pair
        u += units;
        int start = 0;                           // the pair that holds unit u0, 32 looked at together
        while (start < pairs) {
          int inc = start + lane < pairs ? pair_of(p, s, (start + lane) * kPairRows).tiles + kSegmentCost : 0;
          const int own = inc;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
          }
          const unsigned past = __ballot_sync(0xffffffffu, begin + int64_t(inc) * p.n_kv_heads > u0);
          if (past) {
            const int f = __ffs(past) - 1;
            begin += int64_t(__shfl_sync(0xffffffffu, inc - own, f)) * p.n_kv_heads;
            start += f;
            break;
          }
          begin += int64_t(__shfl_sync(0xffffffffu, inc, 31)) * p.n_kv_heads;
          start += 32;
        }
        for (int pr = start; pr < pairs && begin < u1 && ok; ++pr) {
          const Pair pa = pair_of(p, s, pr * kPairRows);
          const int span = pa.tiles + kSegmentCost;      // the item's units: its cost, then its tiles
          const int64_t width = int64_t(span) * p.n_kv_heads;
          int head = u0 > begin ? int((u0 - begin) / span) : 0;
          for (; head < p.n_kv_heads && begin + int64_t(head) * span < u1 && ok; ++head) {
            const int64_t first = begin + int64_t(head) * span + kSegmentCost, end = first + pa.tiles;
            const int v0 = int(max(u0 - first, int64_t(0))), v1 = int(min(u1 - first, int64_t(pa.tiles)));
            if (v1 <= v0) continue;
            // a part that starts its item goes to the CTA's second place, one that continues it to the first
            const int dest = v0 == 0 && v1 == pa.tiles ? -1 : int(2 * blockIdx.x) + (v0 == 0);
            if (v0 == 0 && v1 < pa.tiles) {
              join.last = int((end - 1) / per);
              join.slot = dest;
              join.t0 = s.t0;
              join.row0 = pr * kPairRows;
              join.rows = min(kPairRows, rows - join.row0);
              join.head = head;
            }
            // each half's first and last tile of the segment
            int lo[2] = {INT32_MAX, INT32_MAX}, hi[2] = {-1, -1};
            auto tile_of = [&](int v) { return v < pa.sink_tiles ? v : v - pa.sink_tiles + pa.w0; };
            auto sees = [&](int x, int v) {
              const int t = tile_of(v);
              return t <= pa.hi[x] && (t >= pa.lo[x] || int64_t(t) * kTile < p.sinks);
            };
            for (int x = 0; x < 2; ++x) {
              for (int v = v0 + lane; v < v1; v += 32)
                if (sees(x, v)) {
                  lo[x] = min(lo[x], v);
                  hi[x] = max(hi[x], v);
                }
              lo[x] = __reduce_min_sync(0xffffffffu, lo[x]);
              hi[x] = __reduce_max_sync(0xffffffffu, hi[x]);
            }
            // lane i: block i of the keys, lane 8 + i: of the values; a tile's page ids load while the one before
            // it is handed out
            auto id_of = [&](int v) {
              const int blk = tile_of(v) * kTile + (lane & 7) * kBlock;
              return v < v1 && lane < 16 && blk < s.len ? table[blk / a.page_size] : -1;
            };
            int id = id_of(v0);
            for (int v = v0; v < v1; ++v, ++it) {
              const int mi = it % kMetaSlots, pos = tile_of(v) * kTile;
              const int id_next = id_of(v + 1);
              int flags = (v == v0 ? kBegin : 0) | (v == v1 - 1 ? kEnd : 0);
              for (int x = 0; x < 2; ++x) {
                if (hi[x] >= 0) flags |= x ? kHas1 : kHas0;
                if (sees(x, v)) flags |= x ? kAct1 : kAct0;
                if (v == lo[x]) flags |= x ? kBegin1 : kBegin0;
                if (v == hi[x]) flags |= x ? kEnd1 : kEnd0;
              }
              const bool keys = flags & (kAct0 | kAct1);
              const int blk = pos + (lane & 7) * kBlock;
              int page = -1;
              if (keys && lane < 16 && blk < s.len) page = checked_page(a, id, err);
              id = id_next;
              const unsigned here = __ballot_sync(0xffffffffu, page >= 0);
              const unsigned missing = __ballot_sync(0xffffffffu, keys && lane < 8 && blk < s.len && page < 0);
              if (missing) flags |= kHoles;
              if (!wait(&sh.meta_empty[mi], ((it / kMetaSlots) & 1) ^ 1)) {
                ok = false;
                break;
              }
              PreMeta& me = sh.meta[mi];
              const int off = blk % a.page_size;
              if (lane < 16) {
                float* dst = lane < 8 ? &me.ks[lane] : &me.vs[lane & 7];
                if (page >= 0) {
                  const float* sc = (lane < 8 ? p.k_scales : p.v_scales) + int64_t(page) * p.scale_stride +
                                    head * (a.page_size / kBlock) + off / kBlock;
                  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(sc) : "memory");
                } else {
                  *dst = 1.0f;
                }
              }
              asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.meta_full[mi]))
                           : "memory");
              if (lane == 0) {
                me.pos = pos;
                me.flags = flags;
                me.t0 = s.t0;
                me.row0 = pr * kPairRows;
                me.rows = min(kPairRows, rows - me.row0);
                me.past = s.past;
                me.head = head;
                me.dest = dest;
                me.missing = missing;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.meta_full[mi]);
              if (!keys) continue;
              for (int kv = 0; kv < 2; ++kv, ++n) {
                const int rs = n % kRawSlots;
                if (!wait(&sh.raw_empty[rs], ((n / kRawSlots) & 1) ^ 1)) {
                  ok = false;
                  break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&sh.raw_full[rs], __popc(here & (kv ? 0xff00u : 0xffu)) * kBlock * D);
                __syncwarp();
                if (page >= 0 && (lane >> 3) == kv)
                  tma_load_4d(sh.raw[rs] + (lane & 7) * kBlock * D, kv ? &map_v : &map_k, 0, off, head, page,
                              &sh.raw_full[rs]);
              }
              if (!ok) break;
            }
          }
          begin += width;
        }
      }
    }
    if (lane == 0) p.joins[blockIdx.x] = join;
    if (ok) {
      const int mi = it % kMetaSlots;
      if (wait(&sh.meta_empty[mi], ((it / kMetaSlots) & 1) ^ 1)) {
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.meta_full[mi]))
                     : "memory");
        if (lane == 0) {
          sh.meta[mi].flags = kStop;
          mbar_arrive(&sh.meta_full[mi]);
        }
      }
    }
    // every copy issued has landed before the CTA's shared memory goes
    for (int i = max(0, n - kRawSlots); i < n; ++i)
      drain(&sh.raw_full[i % kRawSlots], (i / kRawSlots) & 1);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kSoftmaxWarps + kWidenWarps + 1) {
    // ----------------------------------------------------------- the products
    // QK of a tile is issued one tile ahead of its PV, interleaved by row tile:
    // S0(j+1) right behind O0(j), while softmax 1 works on tile j.
    if (elect_one()) {
    auto wait1 = [&](uint64_t* bar, uint32_t parity) { return wait_small(bar, parity, p.wait, abort, err); };
    // bit x: parity of the row tile's next q rows, weights, free O; whether its O was used before (bits, because an
    // array indexed by x would live in local memory)
    uint32_t q_ph = 0, p_ph = 0, of_ph = 0, used_o = 0;
    int n = 0;                                   // code tiles taken
    bool ok = true;
    // S = Q K^T of row tile x
    auto product_s = [&](int x, int hs, int flags) {
      if (flags & (x ? kBegin1 : kBegin0)) {
        if (!wait1(&sh.q_full[x], (q_ph >> x) & 1)) return false;
        q_ph ^= 1u << x;
      }
      tc_after();
      const uint64_t q = desc_k(smem_u32(sh.q[x])), k = desc_k(smem_u32(sh.half[hs]));
      const uint32_t d = tmem + x * kTile;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          constexpr int kStep = 32 >> 4;         // 16 channels, in the descriptor's units
          const int o = (i >> 2) * (kTile * 128 >> 4) + (i & 3) * kStep;
          tc_mma_ss(d, q + o, k + o, kIdescS, i > 0);
        }
        tc_commit(&sh.s_full[x]);
        if (flags & (x ? kEnd1 : kEnd0)) tc_commit(&sh.q_free[x]);
      return true;
    };
    auto product_o = [&](int x, int hs, int flags) {
      if (!wait1(&sh.p_ready[x], (p_ph >> x) & 1)) return false;
      p_ph ^= 1u << x;
      if (flags & (x ? kBegin1 : kBegin0)) {
        if ((used_o >> x) & 1) {
          if (!wait1(&sh.o_free[x], (of_ph >> x) & 1)) return false;
          of_ph ^= 1u << x;
        }
        used_o |= 1u << x;
      }
      tc_after();
      const uint64_t v = desc_mn(smem_u32(sh.half[hs]));
      const uint32_t more = (flags & (x ? kBegin1 : kBegin0)) ? 0u : 1u;
      const uint32_t d = tmem + 2 * kTile + x * D, w = tmem + x * kTile;
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i) 
          tc_mma_ts(d, w + (i >> 2) * (kTile / 2) + (i & 3) * 8, v + i * (2048 >> 4), kIdescO, i > 0 ? 1u : more);
        tc_commit(&sh.o_full[x]);
      return true;
    };
    // the flags of the next tile with keys (0: none left)
    int it = 0;
    auto take = [&]() -> int {
      for (;;) {
        const int mi = it % kMetaSlots;
        if (!wait1(&sh.meta_full[mi], (it / kMetaSlots) & 1)) return -1;
        const int f = sh.meta[mi].flags;
        if (f & kStop) return 0;
        ++it;
        mbar_arrive(&sh.meta_empty[mi]);
        if (f & (kAct0 | kAct1)) return f;
      }
    };
    // A round: O of the tile at hand (none in the first round), S of the next (none in the last). Within a segment
    // in the order O0, S0, O1, S1; where the next tile begins one, both O first: its q rows may still be on the way.
    for (int cur = 0;;) {
      const int next = take();
      if (next < 0 || (next == 0 && cur == 0)) break;
      const int vs = n % kHalfSlots;
      if (cur) {
        ok = wait1(&sh.half_full[vs], (n / kHalfSlots) & 1);
        ++n;
      }
      const int ks = n % kHalfSlots;
      const uint32_t k_ph = (n / kHalfSlots) & 1;
      const bool same = !(next & kBegin);
      bool have_k = false;
#pragma unroll 1
      for (int step = 0; step < 4 && ok; ++step) {
        const int x = same ? step >> 1 : step & 1;
        const int bit = x ? kAct1 : kAct0;
        if (!(same ? step & 1 : step >> 1)) {
          if (cur & bit) ok = product_o(x, vs, cur);
          if (ok && cur && x == 1) tc_commit(&sh.half_empty[vs]);
        } else if (next & bit) {
          if (!have_k) ok = wait1(&sh.half_full[ks], k_ph);
          have_k = true;
          if (ok) ok = product_s(x, ks, next);
        }
      }
      if (!ok || next == 0) break;
      tc_commit(&sh.half_empty[ks]);
      ++n;
      cur = next;
    }
    // everything issued has finished before tensor memory is given back
    tc_commit(&sh.done);
    drain(&sh.done, 0);
    }
  } else {
    // ------------------------------------------------------------------ q rows
    // Each warp brings 64 rows of both tiles: asynchronous copies into their swizzled places, then, for bf16, a
    // turn in place to fp16 over a power of two of the row's largest magnitude.
    constexpr int CPR = D / 8;                   // 16-byte chunks of a row
    const int r_first = (warp - (kSoftmaxWarps + kWidenWarps + 2)) * 64;
    uint32_t q_ph[2] = {0, 0}, seg = 0;
    int used[2] = {0, 0};
    for (int it = 0;; ++it) {
      const int mi = it % kMetaSlots;
      if (!wait(&sh.meta_full[mi], (it / kMetaSlots) & 1)) break;
      const PreMeta& me = sh.meta[mi];
      const int flags = me.flags, t0 = me.t0, row0 = me.row0, rows = me.rows, head = me.head;
      if (flags & kStop) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.meta_empty[mi]);
      bool ok = true;
      if (flags & kBegin) {
        for (int x = 0; x < 2 && ok; ++x) {
          if (!(flags & (x ? kHas1 : kHas0))) continue;
          if (used[x]++) {
            ok = __all_sync(0xffffffffu, wait_small<true>(&sh.q_free[x], q_ph[x], p.wait, abort, err));
            q_ph[x] ^= 1;
            if (!ok) break;
          }
          const uint32_t dst = smem_u32(sh.q[x]);
          // lane i: where rows i and 32 + i of this warp's lie
          int64_t at[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int gr = row0 + x * kTile + r_first + 32 * k + lane, tok = gr / p.group;
            at[k] = int64_t(t0 + tok) * p.q_stride + int64_t(head * p.group + gr - tok * p.group) * D;
          }
#pragma unroll 4
          for (int i = lane; i < 64 * CPR; i += 32) {
            const int k = i / CPR, r = r_first + k, c = i % CPR;
            const int64_t off = __shfl_sync(0xffffffffu, i < 32 * CPR ? at[0] : at[1], k & 31);
            const bool there = x * kTile + r < rows;
            const uint16_t* src = there ? p.q + off + c * 8 : p.q;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             dst + (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                         "l"(src), "r"(there ? 16 : 0)
                         : "memory");
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        for (int x = 0; x < 2 && ok; ++x) {
          if (!(flags & (x ? kHas1 : kHas0))) continue;
          if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll 1
            for (int r = r_first + lane; r < r_first + 64; r += 32) {
              uint8_t* src = sh.q[x] + r * 128;
              auto chunk = [&](int c) {
                return reinterpret_cast<uint4*>(src + (c >> 3) * (kTile * 128) + (((c & 7) ^ (r & 7)) << 4));
              };
              float top = 0.0f;
#pragma unroll 4
              for (int c = 0; c < CPR; ++c) {
                float y[8];
                unpack8<T>(*chunk(c), y);
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(y[j]));
              }
              const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
              const float inv = __uint_as_float((254u - e) << 23);
              sh.factor[seg % kMetaSlots][x][r] = __uint_as_float(e << 23);
#pragma unroll 4
              for (int c = 0; c < CPR; ++c) {
                float y[8];
                unpack8<T>(*chunk(c), y);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] *= inv;
                *chunk(c) = pack8<__half>(y);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.q_full[x]);
        }
      }
      if (flags & kEnd) ++seg;
      if (!ok) break;
    }
  }

  tc_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + kWidenWarps + 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Joins the parts of the item that starts in CTA blockIdx.x's run, 32 rows to
// a block: lane = row, a warp the channels 4 w .. of each 32; parts in order.
template <typename T, int D>
__global__ void __launch_bounds__(256) join_rows_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kRow = D * 2 + 16;
  __shared__ __align__(16) uint8_t tile[32 * kRow];
  pdl_launch();
  pdl_wait();
  const Join j = p.joins[blockIdx.x];
  if (j.last < 0 || int(blockIdx.y) * 32 >= j.rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * 32 + lane;          // (rows behind the item's read what is there and are not written)
  const int c0 = blockIdx.x, n = j.last - c0 + 1;
  auto part = [&](int i) { return p.part + int64_t(i == 0 ? j.slot : 2 * (c0 + i)) * (kPairRows * (D + 2)); };
  float top = -INFINITY, sum = 0.0f;
  const bool mine = r < j.rows;
  for (int i = 0; i < n && mine; ++i) top = fmaxf(top, part(i)[kPairRows * D + 2 * r]);
  float4 o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = 0; i < n && mine; ++i) {
    const float2 st = *reinterpret_cast<const float2*>(part(i) + kPairRows * D + 2 * r);
    const float f = st.x == -INFINITY ? 0.0f : exp2_fast(st.x - top);
    sum = fmaf(f, st.y, sum);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const float4 y = *reinterpret_cast<const float4*>(part(i) + ((e * 8 + warp) * kPairRows + r) * 4);
      o[e].x = fmaf(f, y.x, o[e].x);
      o[e].y = fmaf(f, y.y, o[e].y);
      o[e].z = fmaf(f, y.z, o[e].z);
      o[e].w = fmaf(f, y.w, o[e].w);
    }
  }
  const float inv = inverse(top, sum);
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    *reinterpret_cast<uint2*>(tile + lane * kRow + (e * 8 + warp) * 8) =
        make_uint2(Half16<T>::pack(o[e].x * inv, o[e].y * inv), Half16<T>::pack(o[e].z * inv, o[e].w * inv));
  __syncthreads();
  constexpr int CPR = D / 8;
  for (int i = threadIdx.x; i < 32 * CPR; i += 256) {
    const int q = i / CPR, c = i % CPR, row = j.row0 + blockIdx.y * 32 + q;
    if (int(blockIdx.y) * 32 + q >= j.rows) break;
    *reinterpret_cast<uint4*>(p.out + int64_t(j.t0 + row / p.group) * p.out_stride +
                              int64_t(j.head * p.group + row % p.group) * D + c * 8) =
        *reinterpret_cast<const uint4*>(tile + q * kRow + c * 16);
  }
}

// awq_kv_attention: attention over the 8-bit paged KV cache.
//
// Mathematics. One key / value head serves group = n_q_heads / n_kv_heads
// query heads, so the rows of a sequence and head are the (token, head of the
// group) pairs, R of them to a tile. For a tile of 16 keys (one scale block)
//   S = K_codes q^T            exact products, fp32 sums (tensor cores)
//   t_j = scale log2(e) s_k S_j + log2(s_v)
//   p_j = 2^(t_j - m + 7),  O += V_codes^T p,  l += p_j / s_v
// with a running maximum m of t, and y = O / l at the end: the value scale
// rides on the weight (sum 2^(t'_j) s_v c_j / sum 2^(t'_j), t' = t - log2
// s_v), so the codes enter the second product as they are, and p <= 2^15 fits
// fp16 whatever the scales. m is only raised when a logit passes it by more
// than 8 (then O and l are rescaled); below that p stays within fp16. The lift
// by 2^7 is for long contexts: fp16 holds p down to 2^-25, so what is rounded
// off a weight is at most 2^-32 of the largest's, and n keys lose n 2^-32.
//
// What bounds it: for the few rows of decoding, reading the cache. Both
// products have the codes as the 16-row operand of mma.sync.m16n8k16 (16 keys
// or 16 channels by 16) and the rows as its 8 columns, fed from registers:
// a code is used once per row tile, so writing its 16-bit form to shared
// memory for a tcgen05 operand would cost several times the bytes read from
// HBM, as in the GEMV. The transposition of S into the second product's
// operand is one movmatrix per 8 keys; the channel order of both operands is
// chosen so that a lane's codes are 16 contiguous bytes, and the TMA's
// swizzle makes those reads free of bank conflicts.
//
// Split. All (sequence, row tile, head) items are laid end to end, each as a
// fixed cost and its tiles of 16 keys, and cut into equal runs, one per
// resident CTA, whatever the lengths; the cut is computed by every CTA from
// the lengths in device memory. An item that lies within one CTA's run is
// written out directly. Of an item that spans several, each writes (m, l, O)
// to the workspace, and a second kernel joins them in order; it needs no
// counters, so the workspace carries no state. Where there is a CTA for every
// item and none can be long, items are taken whole and nothing is joined.
//
// In a CTA one producer warp looks up pages and issues the TMA copies (a box
// of 16 tokens x head_dim per copy) and four consumer warps take two 16-key
// tiles of each stage, each with its own m, l and O, joined at the item's end.
//
// Measured on one B200 (a Python call, launches included): 32 sequences of up
// to 8192 tokens, 32 / 8 heads of 128, int8 (276 MB) 59 us, 4.7 TB/s; two of
// up to 131001, 64 / 8 heads, e4m3 (381 MB) 87 us, 4.4 TB/s; 48 sequences of
// 5 rows, 16 heads of 64 (197 MB) 53.5 us, 3.7 TB/s; one of 777 tokens 13.5 us,
// 9 of them on the GPU. The same copies with no arithmetic: 60, 71, 57 us
// before the items' cost was counted (then 71, 91, 77 with it).

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "awq_kv.cuh"
#include "awq_tma_host.h"

namespace awq {
namespace kv {
namespace {

__device__ uint32_t g_kv_attention_error = 0;

constexpr int W = 4;                       // consumer warps
constexpr int kThreads = (W + 1) * 32;
constexpr int U = 2;                       // tiles of a warp in a stage
constexpr int WT = W * U;                  // tiles of a stage
constexpr int kStages = 2;
// What an item costs a CTA beyond its tiles (q rows, the warps' joining, output), in tiles: the cut counts every item as
// that much longer. (On the GPU, 0, 8, 12, 14: 128 sequences of up to 128 tokens 30, 17, 16, 21 us; 32 of up to 2000 32,
// 18, 20, 24, e4m3 and groups of 8 39, 22, 22, 28; 48 sequences of 5 rows over 4000, heads of 64, 64, 48, 54, 51.)
constexpr int kItemCost = 12;
constexpr int kItems = 8;                  // more than the stages in the ring and the one ahead of it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;             // how far a logit may pass m (log2 units)
constexpr float kLift = 7.0f;              // log2 of the weight at m: with kSlack, the largest that fp16 has room for

// How long a pipeline wait lasts before it gives up (awq_debug_set_wait_limit_ns shortens it for tests).
struct WaitLimit {
  uint32_t polls;                          // polls between two looks at the clock; 1: a shortened limit
  long long cycles;
};

struct AttentionParams {
  Batch batch;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_stride, out_stride;
  const float* k_scales;
  const float* v_scales;
  int64_t scale_stride;
  float scale_log2;
  int32_t window, sinks;
  int32_t group, n_kv_heads;
  float inv_group;
  int32_t whole;                           // few rows: a CTA takes whole items (no parts, no join)
  float* part;                             // [2 grid][R][D + 2] fp32
  struct Join* joins;                      // [grid]
  WaitLimit wait;
};

// A split item, described by the CTA in whose run it starts.
struct Join {
  int32_t last;      // CTA in whose run it ends; -1: no such item
  int32_t slot;      // its first part
  int32_t t0, row0, rows, head;
  int32_t pad[2];
};

// The first key in the window of position p.
__device__ __forceinline__ int window_start(int p, int window) { return window && p >= window ? p - window + 1 : 0; }

// The keys that a sequence's rows may see: sink tiles, then the tiles from w0.
struct Span {
  int tiles, sink_tiles, w0, row_tiles;
};

template <int R>
__device__ __forceinline__ Span span_of(const AttentionParams& p, const Seq& s) {
  Span a;
  if (s.n == 0) {
    a.tiles = a.sink_tiles = a.w0 = a.row_tiles = 0;
    return a;
  }
  const int low = window_start(s.past, p.window);
  a.w0 = min(low, s.len) / kBlock;
  a.sink_tiles = p.window ? min((min(p.sinks, low) + kBlock - 1) / kBlock, a.w0) : 0;
  a.tiles = max(a.sink_tiles + (s.len + kBlock - 1) / kBlock - a.w0, 1);   // one for a row that sees nothing
  a.row_tiles = int((int64_t(s.n) * p.group + R - 1) / R);
  return a;
}

template <int D, int R>
struct Shared {
  static constexpr int kTile = kBlock * D;              // bytes of 16 keys or values
  static constexpr int kStageBytes = 2 * WT * kTile;
  struct Meta {
    int tile[WT];           // position of the tile's first key, -1: nothing there
    float ks[WT], vs[WT];
    int flags;
  };
  struct Item {
    int tok0, rem0;         // the token of its first row, and that row's head in the group
    int t0, row0, rows, past, head, dest;
  };
  uint8_t ring[kStages][kStageBytes];
  uint8_t q[kStages][R * D * 2];               // the item's q rows, in its first stage
  float2 stat[2][W][R];                        // [merge parity][warp][row]: m, l
  Meta meta[kStages];
  Item items[kItems];
  uint64_t full[kStages], empty[kStages], merged;
  int64_t scratch[40];
  int abort;
};

// A bounded wait in few instructions: it is inlined in many places, and a
// warp that polls shares its scheduler with one that works. LIMITED: one
// wait of each kernel off its critical path (for a free slot, few rows; for
// the place of the next segment's q rows, many), which a shortened limit makes
// run out; its polls do not sleep then (a poll that sleeps may do so for longer
// than its hint). The others see the abort flag. (With that form in every wait
// the many-row kernel takes 13 % longer, in the few-row consumers' alone 3 %.)
template <bool LIMITED = false>
__device__ __forceinline__ bool wait_small(uint64_t* bar, uint32_t parity, const WaitLimit& limit, volatile int* abort,
                                           uint32_t* err) {
  for (long long t0 = 0;;) {
    uint32_t ok;
    if constexpr (LIMITED) {
      asm volatile(
          "{\n\t.reg .pred p, q, w;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n\tsetp.ne.u32 w, %4, 1;\n"
          "POLL_%=:\n\t@w mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "@!w mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
          "@p bra DONE_%=;\n\tadd.u32 n, n, 1;\n\tsetp.lt.u32 q, n, %4;\n\t@q bra POLL_%=;\n"
          "DONE_%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u), "r"(limit.polls)
          : "memory");
    } else {
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
          "POLL_%=:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "@p bra DONE_%=;\n\tadd.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 256;\n\t@q bra POLL_%=;\n"
          "DONE_%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
          : "memory");
    }
    if (ok) return true;
    const long long t = clock64();
    if (t0 == 0) t0 = t;
    if (t - t0 > (LIMITED ? limit.cycles : 2 * static_cast<long long>(kWaitLimitNs)) || *abort) {
      *abort = 1;
      atomicOr(err, kErrWait);
      return false;
    }
  }
}

// Copies or products under way are waited for before a CTA ends, by the clock
// of the SM (the global timer takes about a microsecond to read).
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  for (const long long t0 = clock64();
       !mbar_try_wait_sleep(bar, parity) && clock64() - t0 < 2 * static_cast<long long>(kWaitLimitNs);) {
  }
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Codes as fp16, exactly but for a power of two (kShift). int8: a byte u under
// 0x64 is the fp16 number 1024 + u = 1152 + code. e4m3: exponent and mantissa
// in the places of fp16's are the number times 2^-8 (the exponents' biases are
// 7 and 15; subnormal numbers too), in half the instructions of a conversion
// by cvt. (The NaN codes, which the cache never gets, come out as 480.)
template <int FMT>
constexpr float kShift = FMT == AWQ_KV_E4M3 ? 256.0f : 1.0f;

// Bytes 0 and 2 of w.
template <int FMT>
__device__ __forceinline__ uint32_t code_even(uint32_t w) {
  if constexpr (FMT == AWQ_KV_INT8) return hsub2_u32(lop3_and_or(w, 0x00ff00ffu, 0x64006400u), 0x64806480u);
  return (w & 0x007f007fu) * 128u + (w & 0x00800080u) * 256u;
}
// Bytes 1 and 3 of w.
template <int FMT>
__device__ __forceinline__ uint32_t code_odd(uint32_t w) {
  if constexpr (FMT == AWQ_KV_INT8) return hsub2_u32(__byte_perm(w, 0x64646464u, 0x4341), 0x64806480u);
  return ((w & 0x7f007f00u) >> 1) | (w & 0x80008000u);
}
// Bytes LO and LO + 1 of w.
template <int FMT, int LO>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  if constexpr (FMT == AWQ_KV_INT8) return hsub2_u32(__byte_perm(w, 0x64646464u, LO ? 0x4342 : 0x4140), 0x64806480u);
  const uint32_t z = __byte_perm(w, 0u, LO ? 0x4342 : 0x4140) * 128u;
  return z + (z & 0x40004000u);
}

// A row of q as the products' column operand: lane (n, t) holds channels
// [D/4 t, D/4 (t + 1)) of row n. bf16 rows are brought to fp16 over a power
// of two of their largest magnitude, returned in `factor` (of row n).
template <typename T, int D>
__device__ __forceinline__ void load_q(const uint8_t* row, int t, uint32_t (&f)[D / 8], float& factor) {
  uint4 raw[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) raw[i] = *reinterpret_cast<const uint4*>(row + t * (D / 2) + i * 16);
  factor = 1.0f;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    float x[D / 32][8], top = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      unpack8<T>(raw[i], x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[i][j]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^e <= top: its exponent field alone, kept where the reciprocal is a normal number too
    const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
    factor = __uint_as_float(e << 23);
    const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] *= inv;
      raw[i] = pack8<__half>(x[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    // channels (0, 2), (1, 3) of each four, as code_even and code_odd give them
    f[4 * i] = __byte_perm(raw[i].x, raw[i].y, 0x5410);
    f[4 * i + 1] = __byte_perm(raw[i].x, raw[i].y, 0x7632);
    f[4 * i + 2] = __byte_perm(raw[i].z, raw[i].w, 0x5410);
    f[4 * i + 3] = __byte_perm(raw[i].z, raw[i].w, 0x7632);
  }
}

template <typename T, int D, int FMT, int NT>
__global__ void __launch_bounds__(kThreads, NT == 2 ? 2 : D == 64 ? 4 : 3)
decode_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ AttentionParams p) {
  constexpr int R = 8 * NT;
  using Sh = Shared<D, R>;
  extern __shared__ uint8_t smem_raw[];
  // (an offset from the array, not a rounded address: the compiler then knows it is shared memory)
  Sh& sh = *reinterpret_cast<Sh*>(smem_raw + ((0u - smem_u32(smem_raw)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &sh.abort;
  uint32_t* err = &g_kv_attention_error;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 33);   // the producer's arrival with the byte count, its lanes' scale copies
      mbar_init(&sh.empty[i], W);
    }
    mbar_init(&sh.merged, W);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  pdl_launch();
  pdl_wait();
  // one answer for the whole warp, so that its collective instructions stay together when a wait gives up
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_small(bar, parity, p.wait, abort, err)) != 0;
  };

  // row / group for the rows of a tile, counted from a token's first (below 2^17: a float's product is exact enough)
  auto by_group = [&](int row) { return int((float(row) + 0.5f) * p.inv_group); };

  // this CTA's run of units
  int64_t per = 0, total = 0, rest = 0;
  const int b_first = locate(
      p.batch.n_seqs, sh.scratch,
      [&](int b) {
        const Span a = span_of<R>(p, load_seq(p.batch, b, err));
        return int64_t(p.whole ? 1 : a.tiles + kItemCost) * a.row_tiles * p.n_kv_heads;
      },
      [&](int64_t sum) {
        per = divide(sum + gridDim.x - 1, gridDim.x);
        return per * blockIdx.x;
      },
      &rest, &total);
  const int64_t u0 = per * blockIdx.x, u1 = min(u0 + per, total);
  __syncthreads();   // the barriers are set up (locate need not have synchronized)

  if (warp == W) {
    // ------------------------------------------------------------ producer
    Join join;
    join.last = -1;
    int s = 0;
    uint32_t ph = 0, used = 0;       // used: stages filled at least once
    if (b_first >= 0) {
      int b = b_first;
      Seq seq = load_seq(p.batch, b, err);
      Span a = span_of<R>(p, seq);
      // An item's units are its cost, then its tiles (whole items: one unit). rel: the current item's first unit,
      // counted from the run's; tile .. end: its tiles of this run.
      const int run = int(u1 - u0), width = p.whole ? 1 : a.tiles + kItemCost;
      int item = int(divide(rest, width)), rel = int(int64_t(item) * width - rest), tile = 0, end = 0;
      int items = a.row_tiles * p.n_kv_heads;
      const int32_t* table = p.batch.table + int64_t(b) * p.batch.table_stride;
      uint32_t n_items = 0;
      bool fresh = true;             // the next stage begins an item, or this run
      bool more = p.whole || max(rel + kItemCost, 0) < run;   // there is a next stage
      const int i = lane % WT;
      // One stage ahead of the copies: the tiles of the next stage, and the loads of its pages' ids. lane i < WT: tile
      // i's keys, lane WT + i: its values. What an item's stages share goes to a ring of its own.
      struct Stage {
        int flags, pos, id;          // flags: first | last << 1 | the run's last << 2 | item's place << 8
      };
      auto next = [&](Stage& st) {
        if (fresh) {
          while (item >= items) {    // on to the next sequence with rows
            seq = load_seq(p.batch, ++b, err);
            a = span_of<R>(p, seq);
            item = 0;
            items = a.row_tiles * p.n_kv_heads;
            table = p.batch.table + int64_t(b) * p.batch.table_stride;
          }
          const int first = rel + kItemCost, row_tile = item / p.n_kv_heads;
          tile = p.whole ? 0 : max(-first, 0);
          end = p.whole ? a.tiles : min(run - first, a.tiles);
          const bool split = tile > 0 || end < a.tiles;
          // a part that starts its item goes to the CTA's second place, one that continues it to the first
          const int dest = split ? int(2 * blockIdx.x) + (tile == 0) : -1;
          ++n_items;
          auto& it = sh.items[n_items % kItems];
          const int row0 = row_tile * R, rows = min(R, seq.n * p.group - row0), head = item - row_tile * p.n_kv_heads;
          const int tok0 = row0 / p.group;
          if (lane == 0) {
            it.tok0 = tok0;
            it.rem0 = row0 - tok0 * p.group;
            it.t0 = seq.t0;
            it.row0 = row0;
            it.rows = rows;
            it.past = seq.past;
            it.head = head;
            it.dest = dest;
          }
          if (split && tile == 0) {
            join.last = int(divide(u0 + first + a.tiles - 1, per));
            join.slot = dest;
            join.t0 = seq.t0;
            join.row0 = row0;
            join.rows = rows;
            join.head = head;
          }
        }
        const int cnt = min(WT, end - tile), v = tile + i, first = fresh;
        tile += cnt;
        fresh = tile == end;
        if (fresh) rel += p.whole ? 1 : a.tiles + kItemCost;
        more = !fresh || (p.whole ? rel < run : rel + kItemCost < run);
        st.flags = first | int(fresh) << 1 | int(!more) << 2 | int(n_items % kItems) << 8;
        st.pos = -1;
        st.id = -1;
        if (lane < 2 * WT && i < cnt) {
          const int pos = (v < a.sink_tiles ? v : v - a.sink_tiles + a.w0) * kBlock;
          if (pos < seq.len) {
            st.pos = pos;
            st.id = table[pos / p.batch.page_size];
          }
        }
        if (fresh) ++item;
      };
      Stage cur = {4, -1, -1}, after;  // (a run that ends within an item's cost: one stage without tiles)
      bool go = true;
      if (more) next(cur);
      while (go) {
        go = more;
        if (go) next(after);
        const bool free_slot = wait_small<true>(&sh.empty[s], ph ^ 1, p.wait, abort, err);
        if (!__all_sync(0xffffffffu, free_slot)) break;
        int page = -1;
        if (cur.pos >= 0) page = checked_page(p.batch, cur.id, err);
        auto& m = sh.meta[s];
        const unsigned here = __ballot_sync(0xffffffffu, page >= 0);
        if (lane < WT) m.tile[i] = page >= 0 ? cur.pos : -1;
        if (lane == 0) m.flags = cur.flags;
        __syncwarp();   // the lanes' entries, before the arrival that publishes them
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], uint32_t(__popc(here)) * Sh::kTile);
        __syncwarp();
        const auto& it = sh.items[cur.flags >> 8];
        if (page >= 0) {
          const bool val = lane >= WT;
          const int off = cur.pos % p.batch.page_size, head = it.head;
          tma_load_4d(&sh.ring[s][(val ? WT * Sh::kTile : 0) + i * Sh::kTile], val ? &map_v : &map_k, 0, off, head, page,
                      &sh.full[s]);
          const float* sc = (val ? p.v_scales : p.k_scales) + int64_t(page) * p.scale_stride +
                            head * (p.batch.page_size / kBlock) + off / kBlock;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(val ? &m.vs[i] : &m.ks[i])), "l"(sc)
                       : "memory");
        }
        if (cur.flags & 1) {             // the item's q rows, zeros behind its last
          constexpr int CPR = D / 8;
          const uint32_t dst = smem_u32(sh.q[s]);
          const int t0 = it.t0 + it.tok0, rem0 = it.rem0, rows = it.rows, head0 = it.head * p.group;
#pragma unroll
          for (int c = lane; c < R * CPR; c += 32) {
            const int r = c / CPR, row = rem0 + r, tok = by_group(row);
            const bool there = r < rows;
            const uint16_t* src = p.q;
            if (there) src += int64_t(t0 + tok) * p.q_stride + int64_t(head0 + row - tok * p.group) * D + (c % CPR) * 8;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + c * 16), "l"(src),
                         "r"(there ? 16 : 0)
                         : "memory");
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.full[s])) : "memory");
        used |= 1u << s;
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
        cur = after;
      }
    }
    if (lane == 0 && !p.whole) p.joins[blockIdx.x] = join;
    // Every copy issued lands before the CTA's shared memory goes: the other warps may have given up on the last ones.
    for (int k = 0; k < kStages; ++k)
      if (used & (1u << k)) drain(&sh.full[k], k < s ? ph : ph ^ 1);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, t = lane & 3;
  constexpr bool kScaled = std::is_same<T, __nv_bfloat16>::value;   // (fp16 rows enter as they are)
  uint32_t qf[NT][D / 8];
  float factor[NT][2];               // of columns 2t, 2t + 1: what q was divided by
  int at[NT][2];                     // positions of those rows
  float m[NT][2], l[NT][2];
  float acc[NT][D / 16][4];
  int p_low = 0, p_high = 0;         // the lowest and highest of them
  int t0 = 0, rem0 = 0, rows = 0, head = 0, dest = 0;   // t0: the token of the item's first row
  int s = 0;
  uint32_t ph = 0, merges = 0;
  for (bool more = b_first >= 0; more;) {
    if (!wait(&sh.full[s], ph)) return;
    const auto& me = sh.meta[s];
    const int flags = me.flags;
    if (flags & 1) {
      const auto& it = sh.items[flags >> 8];
      t0 = it.t0 + it.tok0;
      rem0 = it.rem0;
      rows = it.rows;
      head = it.head;
      dest = it.dest;
      const int past = it.past + it.tok0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mine;
        load_q<T, D>(sh.q[s] + (nt * 8 + g) * (D * 2), t, qf[nt], mine);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (kScaled) factor[nt][e] = __shfl_sync(0xffffffffu, mine, (2 * t + e) * 4);
          at[nt][e] = past + by_group(rem0 + nt * 8 + 2 * t + e);
          m[nt][e] = -INFINITY;
          l[nt][e] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][j][e] = 0.0f;
      }
      p_low = past;
      p_high = past + by_group(rem0 + rows - 1);
    }
    // N tiles of the warp together, W apart: their loads, products and exponentials overlap. Where the stage has
    // only some of them the others' weights are 0 (one path for all keeps the code in the instruction cache).
    auto take = [&](auto count, int first) {
      constexpr int N = decltype(count)::value;
      // (not the first alone: its page may be missing and the next one's there)
      bool any = false;
#pragma unroll
      for (int u = 0; u < N; ++u) any |= me.tile[first + u * W] >= 0;
      if (!any) return;
      const uint8_t* kt[N];
      const uint8_t* vt[N];
      int tile[N];
      float ks[N], lv[N], iv[N];
      uint32_t held[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int i = first + u * W;
        kt[u] = &sh.ring[s][i * Sh::kTile];
        vt[u] = &sh.ring[s][(WT + i) * Sh::kTile];
        tile[u] = me.tile[i];
        const bool there = tile[u] >= 0;
        ks[u] = there ? me.ks[i] : 0.0f;
        const float to_log2 = p.scale_log2 * kShift<FMT>;   // (not into factor, which may be 2^126: keys of 0 have logits of 0)
        float vs = there ? me.vs[i] : 1.0f;
        // a scale that is no finite number of at least 0 makes NaN of the logits, which the rows that do not see the
        // block mask (an infinite one times a negative S would be a weight of 0 instead)
        const bool fine = ks[u] >= 0.0f && vs >= 0.0f && ks[u] + vs < INFINITY;
        // values of scale 0 (or below the smallest, which would leave fp32's range here) are 0 whatever their codes: no
        // weight in O; in l they have their keys', by the smallest scale
        held[u] = vs < kScaleFloor ? 0u : ~0u;
        vs = fmaxf(vs, kScaleFloor);
        ks[u] *= to_log2;
        lv[u] = fine ? __log2f(vs) : __int_as_float(0x7fffffff);
        iv[u] = fine ? __fdividef(1.0f / kShift<FMT>, vs) : 0.0f;   // (O holds codes / kShift)
      }
      // S = K q^T
      float sc[N][NT][4];
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[u][nt][0] = sc[u][nt][1] = sc[u][nt][2] = sc[u][nt][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int c = D == 128 ? ((2 * t + i) ^ g) << 4 : (t ^ (g >> 1)) << 4;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const uint4 lo = *reinterpret_cast<const uint4*>(kt[u] + g * D + c);
          const uint4 hi = *reinterpret_cast<const uint4*>(kt[u] + (g + 8) * D + c);
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a[4] = {code_even<FMT>(wl[w]), code_even<FMT>(wh[w]), code_odd<FMT>(wl[w]),
                                   code_odd<FMT>(wh[w])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(sc[u][nt], a, qf[nt][8 * i + 2 * w], qf[nt][8 * i + 2 * w + 1]);
          }
        }
      }
      // weights
      bool raise = false;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const bool all = tile[u] >= 0 && tile[u] + kBlock - 1 <= p_low &&
                         (p.window == 0 || tile[u] > p_high - p.window || tile[u] + kBlock <= p.sinks);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[u][nt][e] = fmaf(sc[u][nt][e], kScaled ? factor[nt][e & 1] * ks[u] : ks[u], lv[u]);
        if (!all) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = tile[u] + g + (e & 2) * 4, q = at[nt][e & 1];
              if (!(tile[u] >= 0 && j <= q && (p.window == 0 || j > q - p.window || j < p.sinks)))
                sc[u][nt][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) raise |= fmaxf(sc[u][nt][e], sc[u][nt][e + 2]) > m[nt][e] + kSlack;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = m[nt][e];
#pragma unroll
            for (int u = 0; u < N; ++u) v = fmaxf(v, fmaxf(sc[u][nt][e], sc[u][nt][e + 2]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float f = v == -INFINITY ? 1.0f : exp2_fast(m[nt][e] - v);
            m[nt][e] = v;
            l[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              acc[nt][j][e] *= f;
              acc[nt][j][e + 2] *= f;
            }
          }
      }
      uint32_t b0[N][NT], b1[N][NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float base[2] = {m[nt][0] == -INFINITY ? 0.0f : m[nt][0] - kLift,
                               m[nt][1] == -INFINITY ? 0.0f : m[nt][1] - kLift};
#pragma unroll
        for (int u = 0; u < N; ++u) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = exp2_fast(sc[u][nt][e] - base[e & 1]);
          l[nt][0] = fmaf(w[0] + w[2], iv[u], l[nt][0]);
          l[nt][1] = fmaf(w[1] + w[3], iv[u], l[nt][1]);
          b0[u][nt] = transpose8x8(Half16<__half>::pack(w[0], w[1])) & held[u];
          b1[u][nt] = transpose8x8(Half16<__half>::pack(w[2], w[3])) & held[u];
        }
      }
      // O += V^T p: lane (g, t) holds channels [D/8 g, D/8 (g + 1)) of keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
      for (int u = 0; u < N; ++u) {
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * t + (i & 1) + (i >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(vt[u] + r * 128 + ((g ^ (r & 7)) << 4));
            vw[i][0] = x.x;
            vw[i][1] = x.y;
            vw[i][2] = x.z;
            vw[i][3] = x.w;
          } else {
            const uint2 x =
                *reinterpret_cast<const uint2*>(vt[u] + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
            vw[i][0] = x.x;
            vw[i][1] = x.y;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          // two channels of two keys to a word
          const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), y0 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
          const uint32_t x1 = __byte_perm(vw[2][w], vw[3][w], 0x5410), y1 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
          const uint32_t a0[4] = {code_even<FMT>(x0), code_odd<FMT>(x0), code_even<FMT>(x1), code_odd<FMT>(x1)};
          const uint32_t a1[4] = {code_even<FMT>(y0), code_odd<FMT>(y0), code_even<FMT>(y1), code_odd<FMT>(y1)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816(acc[nt][2 * w], a0, b0[u][nt], b1[u][nt]);
            mma_16816(acc[nt][2 * w + 1], a1, b0[u][nt], b1[u][nt]);
          }
        }
      }
    };
    // (two tiles of two column groups would not fit the registers)
    constexpr int N = NT == 1 ? U : 1;
#pragma unroll 1
    for (int u = 0; u < U; u += N) take(std::integral_constant<int, N>{}, warp + u * W);
    if (flags & 2) {
      // The item's end: the warps join their parts, each in the place of its own tiles of this stage (four rows to a
      // tile), which is given back when all have read them.
      // (16-byte chunks of rows 2k and 2k + 1 are in the order c ^ k, which spreads a store over the banks)
      auto part = [&](int w, int r, int d) {
        return reinterpret_cast<float*>(&sh.ring[s][((r >> 3) * WT + w + ((r >> 2) & 1) * W) * Sh::kTile]) + (r & 3) * D +
               (d ^ (((r >> 1) & 3) << 2));
      };
      float2(*stat)[R] = sh.stat[merges & 1];
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * t + e;
          float sum = l[nt][e];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          if (g == 0) stat[warp][r] = make_float2(m[nt][e], sum);
          if (r < rows) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
              *reinterpret_cast<float2*>(part(warp, r, D / 8 * g + 2 * j)) = make_float2(acc[nt][j][e], acc[nt][j][e + 2]);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.merged);
      if (!wait(&sh.merged, merges & 1)) return;
      ++merges;
      for (int i = threadIdx.x; i < rows * (D / 4); i += W * 32) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, stat[w][r].x);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float f = top == -INFINITY ? 0.0f : exp2_fast(stat[w][r].x - top);
          const float4 x = *reinterpret_cast<const float4*>(part(w, r, d));
          sum = fmaf(f, stat[w][r].y, sum);
          o.x = fmaf(f, x.x, o.x);
          o.y = fmaf(f, x.y, o.y);
          o.z = fmaf(f, x.z, o.z);
          o.w = fmaf(f, x.w, o.w);
        }
        if (dest < 0) {
          const float inv = top == -INFINITY ? 0.0f : __fdiv_rn(1.0f, sum);
          const int row = rem0 + r, tok = by_group(row);
          uint16_t* dst = p.out + int64_t(t0 + tok) * p.out_stride + int64_t(head * p.group + row - tok * p.group) * D + d;
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(Half16<T>::pack(o.x * inv, o.y * inv), Half16<T>::pack(o.z * inv, o.w * inv));
        } else {
          float* out = p.part + int64_t(dest) * (R * (D + 2));
          *reinterpret_cast<float4*>(out + r * D + d) = o;
          if (d == 0) *reinterpret_cast<float2*>(out + R * D + 2 * r) = make_float2(top, sum);
        }
      }
      fence_proxy_async_smem();   // the next copy comes behind these writes and reads
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[s]);
    more = !(flags & 4);
    if (++s == kStages) {
      s = 0;
      ph ^= 1;
    }
  }
}

constexpr int kJoinThreads = 128;
constexpr int kJoinRows = 4;               // CTAs along y: rows r, r + 4, ...

// Joins the parts of the item that starts in CTA blockIdx.x's run: part
// `slot`, then the first part of each CTA up to `last`. A row's parts are
// taken in turn by GR groups of threads (one pass, with a running maximum, so
// that all loads go out together), which then meet.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int Q = D / 4;                 // threads along a row
  constexpr int GR = kJoinThreads / Q;
  __shared__ float4 sums[GR][Q];
  __shared__ float2 stats[GR];
  pdl_launch();
  pdl_wait();
  const Join j = p.joins[blockIdx.x];
  if (j.last < 0) return;
  const int c0 = blockIdx.x, n = j.last - c0 + 1;
  const int gr = threadIdx.x / Q, d = threadIdx.x % Q;
  for (int r = blockIdx.y; r < j.rows; r += kJoinRows) {
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = gr; i < n; i += GR) {
      const float* part = p.part + int64_t(i == 0 ? j.slot : 2 * (c0 + i)) * (R * (D + 2));
      const float2 st = *reinterpret_cast<const float2*>(part + R * D + 2 * r);
      const float4 x = *reinterpret_cast<const float4*>(part + r * D + 4 * d);
      const float top = fmaxf(m, st.x), base = top == -INFINITY ? 0.0f : top;
      const float f = exp2_fast(m - base), g = exp2_fast(st.x - base);
      m = top;
      l = fmaf(l, f, g * st.y);
      o.x = fmaf(o.x, f, g * x.x);
      o.y = fmaf(o.y, f, g * x.y);
      o.z = fmaf(o.z, f, g * x.z);
      o.w = fmaf(o.w, f, g * x.w);
    }
    sums[gr][d] = o;
    if (d == 0) stats[gr] = make_float2(m, l);
    __syncthreads();
    if (gr == 0) {
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < GR; ++i) top = fmaxf(top, stats[i].x);
      const float base = top == -INFINITY ? 0.0f : top;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        const float f = exp2_fast(stats[i].x - base);
        const float4 x = sums[i][d];
        sum = fmaf(f, stats[i].y, sum);
        o.x = fmaf(f, x.x, o.x);
        o.y = fmaf(f, x.y, o.y);
        o.z = fmaf(f, x.z, o.z);
        o.w = fmaf(f, x.w, o.w);
      }
      const float inv = top == -INFINITY ? 0.0f : __fdiv_rn(1.0f, sum);
      const int row = j.row0 + r;
      uint16_t* dst = p.out + int64_t(j.t0 + row / p.group) * p.out_stride +
                      int64_t(j.head * p.group + row % p.group) * D + 4 * d;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(Half16<T>::pack(o.x * inv, o.y * inv), Half16<T>::pack(o.z * inv, o.w * inv));
    }
    __syncthreads();
  }
}

#include "awq_kv_prefill.cuh"

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
using DecodeFn = void (*)(CUtensorMap, CUtensorMap, AttentionParams);
using JoinFn = void (*)(AttentionParams);

// kind 0, 1: tiles of 8 / 16 rows; 2: pairs of row tiles of 128.
struct Variant {
  DecodeFn main;
  JoinFn join;
  int R, smem, threads;
  dim3 join_grid;         // y and z of it
  int join_threads;
};

template <typename T, int D, int FMT>
Variant variant_of(int kind) {
  if (kind == 0)
    return {decode_attention_kernel<T, D, FMT, 1>, join_kernel<T, D, 8>, 8, int(sizeof(Shared<D, 8>)) + 1024, kThreads,
            dim3(1, kJoinRows), kJoinThreads};
  if (kind == 1)
    return {decode_attention_kernel<T, D, FMT, 2>, join_kernel<T, D, 16>, 16, int(sizeof(Shared<D, 16>)) + 1024,
            kThreads, dim3(1, kJoinRows), kJoinThreads};
  return {prefill_attention_kernel<T, D, FMT>, join_rows_kernel<T, D>, kPairRows, int(sizeof(PreShared<D>)) + 1024,
          kPreThreads, dim3(1, kPairRows / 32), 256};
}

template <typename T>
Variant variant_of(int d, int fmt, int kind) {
  if (d == 128)
    return fmt == AWQ_KV_INT8 ? variant_of<T, 128, AWQ_KV_INT8>(kind) : variant_of<T, 128, AWQ_KV_E4M3>(kind);
  return fmt == AWQ_KV_INT8 ? variant_of<T, 64, AWQ_KV_INT8>(kind) : variant_of<T, 64, AWQ_KV_E4M3>(kind);
}

// The kernel's shared memory limit raised and its resident CTAs counted, once
// per kernel and device.
awq_status_t resident(const Variant& v, int key, int* grid) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[24][kDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return AWQ_ERR_CUDA;
  const bool keep = dev < kDevices;
  int n = keep ? known[key][dev].load(std::memory_order_acquire) : 0;
  if (n == 0) {
    int sms = 0, per_sm = 0;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(v.main), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             v.smem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, reinterpret_cast<const void*>(v.main), v.threads,
                                                      v.smem) != cudaSuccess ||
        per_sm < 1) {
      cudaGetLastError();
      return AWQ_ERR_CUDA;
    }
    n = sms * per_sm;
    if (keep) known[key][dev].store(n, std::memory_order_release);
  }
  *grid = n;
  return AWQ_OK;
}

// What awq_debug_set_wait_limit_ns asks for, on every device.
std::atomic<uint64_t> g_wait_limit_ns{kWaitLimitNs};

WaitLimit wait_limit() {
  const uint64_t ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  return {ns == kWaitLimitNs ? 256u : 1u, 2 * static_cast<long long>(ns)};   // about two cycles a nanosecond
}

size_t workspace_of(const Variant& v, int grid, int d) {
  return size_t(grid) * sizeof(Join) + size_t(grid) * 2 * v.R * (d + 2) * sizeof(float);
}

// The kernel, by the rows (tokens x group) of the longest sequence and the (rows of the call) x (tiles of 16 keys that
// fit a sequence): tiles of 8 rows while they fit one; beyond, tiles of 16, which read the cache once each but start
// fast and share the work finely, until the pairs of 128 on the tensor cores win. Measured on the GPU (tiles of 16 and
// pairs of 128, us; the product of rows and tiles in brackets):
//   32 / 8 heads of 128, int8: 60 tokens of a prompt of 60, 2000, 8000 [1200, 30960, 120240] 7 and 15, 24 and 28, 59
//   and 41; prompts of 128, 256, 512 [4608, 17408, 67584] 8.5 and 15, 22 and 22, 47 and 27. e4m3: within 15 % of these.
//   16 heads of 64, group 1, int8: prompts of 128, 256, 512 [1152, 4352, 16896] 6 and 11, 8 and 15, 23 and 19
//   16 key heads of 64, group 4, e4m3: prompts of 128, 256, 512 [4608, 17408, 67584] 14 and 14, 25 and 20, 65 and 27
// The border lies higher with few key heads and lower with many short sequences, which the rule does not know:
//   1 key head of 128, group 8: 60 tokens of 8000 [240480] 25 and 71, prompts of 512 [135168] 14 and 22
//   8 prompts of 100, 32 / 8 heads [28800] 35 and 17; 16 / 16 heads of 64 [7200] 19 and 13
int kind_of(int64_t rows, int64_t all, int64_t tiles) { return rows <= 8 ? 0 : rows <= 64 || all * tiles <= 32768 ? 1 : 2; }

awq_status_t check_attention(const awq_kv_cache_t* cache, const awq_kv_batch_t* batch, int64_t n_tokens,
                             int32_t n_q_heads) {
  awq_status_t st;
  if ((st = check_cache(cache)) != AWQ_OK || (st = check_batch(batch, n_tokens)) != AWQ_OK ||
      (st = check_capacity(cache, batch)) != AWQ_OK)
    return st;
  if (n_q_heads < 1 || n_q_heads > 65536 || n_q_heads % cache->n_kv_heads) return AWQ_ERR_SHAPE;
  if (n_tokens * (n_q_heads / cache->n_kv_heads) > INT32_MAX / 2) return AWQ_ERR_SHAPE;
  return AWQ_OK;
}

struct Plan {
  Variant v;
  bool many, whole;
  int grid;
};

// Up to how many tiles an item is taken whole by one CTA, without parts and the kernel that joins them, when there is
// a CTA for every item. The tiles are those that the table has room for: with a table of 131072 tokens nothing is taken
// whole. Measured on the GPU (32 / 8 heads of 128, int8; whole and split, us):
//   1 sequence of 128, 500, 1000 tokens:   5.6 and 7.6, 9.5 and 7.9, 15 and 10
//   8 sequences of up to 128, 500, 1000:   6.6 and 8.8, 10 and 12, 16 and 12
//   32 sequences of up to 128, 500, 1000:  7.7 and 9.4, 12.8 and 12.1, 19 and 20
int whole_tiles(int64_t items, int grid) { return items > grid ? 0 : items * 2 >= grid ? 64 : items * 8 >= grid ? 40 : 24; }

awq_status_t plan_of(const awq_kv_cache_t* cache, const awq_kv_batch_t* batch, int64_t n_tokens, int32_t dtype,
                     int32_t n_q_heads, Plan* plan) {
  const int group = n_q_heads / cache->n_kv_heads;
  const int64_t most = batch->max_q_len > 0 && batch->max_q_len < n_tokens ? batch->max_q_len : n_tokens;
  const int64_t tiles = int64_t(batch->max_pages) * (cache->page_size / kBlock) + 1;   // of the longest sequence that fits
  const int kind = kind_of(most * group, n_tokens * group, tiles);
  plan->v = dtype == AWQ_KV_FP16 ? variant_of<__half>(cache->head_dim, cache->format, kind)
                                 : variant_of<__nv_bfloat16>(cache->head_dim, cache->format, kind);
  plan->many = kind == 2;
  const int key = (((dtype == AWQ_KV_BF16) * 2 + (cache->head_dim == 128)) * 2 + (cache->format == AWQ_KV_E4M3)) * 3 + kind;
  const awq_status_t st = resident(plan->v, key, &plan->grid);
  if (st != AWQ_OK) return st;
  // No more CTAs than the longest sequences that fit could give work to.
  const int64_t work = plan->many ? (tiles + 7) / 8 * ((n_tokens * group + kPairRows - 1) / kPairRows + batch->n_seqs)
                                  : (tiles + WT - 1) / WT * ((n_tokens * group + plan->v.R - 1) / plan->v.R + batch->n_seqs);
  const int64_t items = ((n_tokens * group + plan->v.R - 1) / plan->v.R + batch->n_seqs) * cache->n_kv_heads;
  plan->whole = !plan->many && tiles <= whole_tiles(items, plan->grid);
  if (plan->whole)
    plan->grid = int(items);
  else if (work <= plan->grid / cache->n_kv_heads)
    plan->grid = int(work > 0 ? work : 1) * cache->n_kv_heads;
  return AWQ_OK;
}

}  // namespace

void attention_set_wait_limit(uint64_t ns) { g_wait_limit_ns.store(ns, std::memory_order_relaxed); }

awq_status_t attention_take_error(uint32_t* word, cudaStream_t s) {
  const uint32_t zero = 0;
  if (cudaMemcpyFromSymbolAsync(word, g_kv_attention_error, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_kv_attention_error, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return AWQ_ERR_CUDA;
  return AWQ_OK;
}

}  // namespace kv
}  // namespace awq

extern "C" awq_status_t awq_kv_attention_workspace_bytes(const awq_kv_cache_t* cache, const awq_kv_batch_t* batch,
                                                         int64_t n_tokens, int32_t n_q_heads, size_t* bytes) {
  using namespace awq;
  using namespace awq::kv;
  if (!bytes) return AWQ_ERR_NULL;
  awq_status_t st = check_attention(cache, batch, n_tokens, n_q_heads);
  if (st != AWQ_OK) return st;
  *bytes = 0;
  if (n_tokens == 0 || batch->n_seqs == 0) return AWQ_OK;
  for (int32_t dtype : {AWQ_KV_FP16, AWQ_KV_BF16}) {
    Plan plan;
    if ((st = plan_of(cache, batch, n_tokens, dtype, n_q_heads, &plan)) != AWQ_OK) return st;
    const size_t need = workspace_of(plan.v, plan.grid, cache->head_dim);
    if (need > *bytes) *bytes = need;
  }
  return AWQ_OK;
}

extern "C" awq_status_t awq_kv_attention(const awq_kv_cache_t* cache, const awq_kv_batch_t* batch, int64_t n_tokens,
                                         int32_t dtype, const uint16_t* q, int64_t q_stride, int32_t n_q_heads,
                                         float scale, int32_t window, int32_t sinks, uint16_t* out, int64_t out_stride,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  using namespace awq;
  using namespace awq::kv;
  awq_status_t st = check_attention(cache, batch, n_tokens, n_q_heads);
  if (st != AWQ_OK) return st;
  if (!check_dtype(dtype)) return AWQ_ERR_UNSUPPORTED;
  const float to_log2 = scale * kLog2e;   // the kernels multiply it by 2^8 (e4m3) and by block scales
  if (window < 0 || sinks < 0 || !(to_log2 > -0x1p119f && to_log2 < 0x1p119f)) return AWQ_ERR_SHAPE;
  if (n_tokens == 0 || batch->n_seqs == 0) return AWQ_OK;
  if ((st = check_pointers(cache, batch)) != AWQ_OK) return st;
  if ((st = check_rows(q, q_stride, n_q_heads, cache->head_dim)) != AWQ_OK ||
      (st = check_rows(out, out_stride, n_q_heads, cache->head_dim)) != AWQ_OK)
    return st;
  Plan plan;
  if ((st = plan_of(cache, batch, n_tokens, dtype, n_q_heads, &plan)) != AWQ_OK) return st;
  if (!workspace || workspace_bytes < workspace_of(plan.v, plan.grid, cache->head_dim)) return AWQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return AWQ_ERR_ALIGN;

  AttentionParams p = {};
  p.batch = make_batch(cache, batch, n_tokens);
  p.q = q;
  p.out = out;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.k_scales = cache->k_scales;
  p.v_scales = cache->v_scales;
  p.scale_stride = cache->scale_stride;
  p.scale_log2 = to_log2;
  // A window that no sequence can outgrow is none (and the kernels' differences of positions stay in 32 bits).
  p.window = int64_t(window) >= int64_t(batch->max_pages) * cache->page_size ? 0 : window;
  p.sinks = p.window ? sinks : 0;
  p.group = n_q_heads / cache->n_kv_heads;
  p.n_kv_heads = cache->n_kv_heads;
  p.whole = plan.whole;
  p.wait = wait_limit();
  p.inv_group = 1.0f / float(p.group);
  p.joins = static_cast<Join*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + size_t(plan.grid) * sizeof(Join));

  // A page's tokens of one head are rows of head_dim bytes; a box is one scale block of them.
  CUtensorMap map_k, map_v;
  const uint64_t D = cache->head_dim;
  const CUtensorMapSwizzle sw = plan.many  ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                           : CU_TENSOR_MAP_SWIZZLE_64B;
  // (an empty cache still gets a map: every page id is then out of range and no copy is issued)
  const uint64_t pages = cache->n_pages > 0 ? cache->n_pages : 1;
  if (!make_tensor_map_4d(&map_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->k_pages, D, cache->page_size,
                          cache->n_kv_heads, pages, D, D * cache->page_size, cache->page_stride, uint32_t(D), kBlock, 1,
                          1, sw) ||
      !make_tensor_map_4d(&map_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->v_pages, D, cache->page_size,
                          cache->n_kv_heads, pages, D, D * cache->page_size, cache->page_stride, uint32_t(D), kBlock, 1,
                          1, sw))
    return AWQ_ERR_CUDA;

  cudaLaunchAttribute attr;
  cudaLaunchConfig_t lc = overlapped(dim3(unsigned(plan.grid)), plan.v.threads, plan.v.smem, stream, &attr);
  cudaError_t e = cudaLaunchKernelEx(&lc, plan.v.main, map_k, map_v, p);
  if (e == cudaSuccess && !plan.whole) {
    lc = overlapped(dim3(unsigned(plan.grid), plan.v.join_grid.y), plan.v.join_threads, 0, stream, &attr);
    e = cudaLaunchKernelEx(&lc, plan.v.join, p);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return AWQ_ERR_CUDA;
  }
  return AWQ_OK;
}

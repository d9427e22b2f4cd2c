// Decode attention over the cache held in 4 bits (format: kv4.cuh): the kernels and their launches.
//
// score(q, k) = sum_j [ s_j sum_{e in j} q_e c_e + m_j sum_{e in j} q_e ]
// o           = sum_t p_t [ s_tj (c_te - 8) + (m_tj + 8 s_tj) ] / sum_t p_t
// with the codes c, scales s and minima m of each group j of 32 elements; both contractions on the matrix
// units (16 tokens x 8 query heads an instruction), the scales of keys on their sums, those of values on
// the codes (eight bits, exact in bf16). Codes need no conversion: four bits under a mask are the bf16
// number code * 2^-133 or 16 times that, subnormal or next to it, which the units take as it is.
//
// Bound by HBM on paper: 160 bytes for a token and KV head of 128. Next to it stands instruction issue:
// an SM has 23 bytes a clock of HBM, so 3.5 instruction lanes for each code; 16 tokens of a head take 418 warp
// instructions, waits among them. 128 rows of 512 .. 8192 tokens, 32 + 32 heads: 405 us, 4.06 TB/s
// (floor 242; the copies alone 268). 57 % of issue slots are used and no pipe is: 16 warps on an SM, each a chain
// of scores, exponentials and values, are few.
//
// Work split: the steps of all (row, group of KV heads) pairs in one line, cut into as many equal ranges as
// CTAs fit on the GPU at once, so long and short rows share them evenly; states of a pair that
// ranges cut are joined by a second kernel, in the order of their tokens. In a CTA a warp takes one KV
// head; with few KV heads several warps share a head's tokens. A step's tokens (32 for each warp) are
// copied whole, all heads of the CTA by neighbouring lanes, into a ring that the warps share: 640 bytes at
// once reach 6.7 TB/s on scattered slots, 80 bytes for each head 3.2 (8 heads of 128; bulk copies of a
// row for each lane cost 25 instructions each). Two CTAs of eight warps: four of four warps read
// half slots, 3 to 5 % slower.
#pragma once
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "host_common.h"
#include "kv4.cuh"
#include "norm_rope.cuh"

namespace rc {
namespace kv4 {

constexpr int kMaxGroup = 16;

struct Range {     // of one CTA: the pairs it shares with others, -1: none
  int row0, hg0, start0, last0;   // begun before it: first and last CTA
  int row1, hg1, last1;           // begun in it and not ended
  int pad;
};
struct Workspace {
  Range* range;   // [ctas]
  float* ml;      // [ctas][2][heads of a group of KV heads][2]: maximum (base 2), sum
  float* o;       // [ctas][2][heads of a group][d]
};
struct Params {
  rc_kv4_decode_args a;
  Workspace w;
  int* status;
  int G;          // query heads of a KV head
  int HG, TS;     // KV heads of a CTA, warps that share a head's tokens
  int tokens, log_tokens;   // of a step: a power of two
  int stride;     // bytes of a slot
  int groups;     // KV heads / HG
  uint64_t wait_ns;   // bound of a wait
};

template <typename T, int D, int NT>
struct Cfg {
  static constexpr int NG = D / 32, RB = kv4_row_bytes(D);
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int QP = F32 ? 3 : 1;     // bf16 parts of a query element
  static constexpr int UNIT = F32 ? 2 : 7;   // scores are summed in 2^-UNIT
  // of a weight: all its 24 bits. Two parts (16 bits) would take 357 us instead of 405 on 128 rows of
  // 512 .. 8192 tokens, 32 + 32 heads, with 0.22 % of bf16 outputs unlike those of 64 bits instead of 0.11
  static constexpr int PP = 3;
  static constexpr int WARPS = NT > 1 || F32 ? 4 : 8;               // of a CTA, at most
  static constexpr int PER_SM = 2;                                  // CTAs of so many warps
  static constexpr int CH = 4 * NG;          // bytes of a copy: a head's row is five
  static constexpr int HALVES = 5;           // of the ring: K or V of a step
  static constexpr int U = 2;                // tiles of 16 tokens of a warp's step
};
// The most warps of the kernels above on an SM.
constexpr int kMaxWarpsPerSm = 16;
constexpr int kSms = 152;
constexpr int kMaxSmem = 112 << 10;   // of a CTA

// Row r of a tile lies at place(r) of its 16 tokens, so that rows whose addresses differ by an odd
// number of 16 bytes for each place are read without conflicts: the lanes of K that go together take two
// (heads of 64: four) rows of 64 (32) bytes, those of V four rows' pieces.
template <int NG>
__device__ __forceinline__ int place(int r) {
  return NG == 4 ? (r & 8) | (r & 1) << 2 | (r >> 1 & 3) : (r & 8) | (r & 3) << 1 | (r >> 2 & 1);
}

// Whether the phase of that parity is complete; a warp that has to wait sleeps up to 20 us before it looks again,
// as it shares its scheduler with those that work. Limits shorter than that are looked at without sleep.
constexpr uint32_t kSleepNs = 20000;
template <bool SLEEP>
__device__ __forceinline__ bool arrived(uint32_t bar, uint32_t parity) {
  uint32_t done;
  if constexpr (SLEEP)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done) : "r"(bar), "r"(parity), "r"(kSleepNs) : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return __all_sync(~0u, done);
}
// The warp waits for a phase, p.wait_ns at most: then it sets the status word, waits for its own copies and
// says false.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, const Params& p) {
  if (arrived<false>(bar, parity)) return true;
  const bool sleep = p.wait_ns >= kSleepNs;
  if (sleep && arrived<true>(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!(sleep ? arrived<true>(bar, parity) : arrived<false>(bar, parity))) {
    if (__any_sync(~0u, global_timer_ns() - t0 > p.wait_ns)) {
      set_status(p.status, kStatusWaitExpired);
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      return false;
    }
  }
  return true;
}

// Bytes between tokens of a stage: an odd number of 16.
__host__ __device__ constexpr int pitch_of(int heads, int row_bytes) {
  return ((heads * row_bytes + 15) / 16 | 1) * 16;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
constexpr uint32_t pow2_bf16x2(int e) { return (uint32_t)(127 + e) << 7 | (uint32_t)(127 + e) << 23; }
constexpr uint32_t kMinus = 0x80008000u;
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// D (16 x 8) = A (16 x 16) B (16 x 8) + C
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a += b, two by two
__device__ __forceinline__ void add4(float* a, const float* b) {
#pragma unroll
  for (int k = 0; k < 4; k += 2)
    unpack2(add2(pack2(a[k], a[k + 1]), pack2(b[k], b[k + 1])), a[k], a[k + 1]);
}
__device__ __forceinline__ void ldmatrix_x2_trans(uint32_t at, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r0), "=r"(r1) : "r"(at) : "memory");
}
template <int N>
__device__ __forceinline__ void load(const char* at, uint32_t (&r)[N]) {
  static_assert(N == 2 || N == 4, "");
  if constexpr (N == 4) {
    const uint4 v = *(const uint4*)at;
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  } else {
    const uint2 v = *(const uint2*)at;
    r[0] = v.x, r[1] = v.y;
  }
}
// the upper and lower halves' next bf16 part: packs and leaves the rest
__device__ __forceinline__ uint32_t take_part(float& lo, float& hi) {
  const uint32_t p = pack2_bf16(lo, hi);
  lo -= bf16lo(p);
  hi -= bf16hi(p);
  return p;
}

__device__ __forceinline__ int steps_of(const Params& p, int len, int req) {
  if (len <= 0 || len > p.a.max_seq_len || req < 0 || req >= p.a.max_reqs) return 0;
  return (len + p.tokens - 1) >> p.log_tokens;
}

// How the line of steps is cut: range c is [total c / ctas, total (c + 1) / ctas).
// Products of 32 bits, the usual case, are divided as such: a 64-bit division takes a few hundred cycles.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
struct Cut {
  int64_t total;
  int ctas;
  __device__ int64_t begin(int c) const { return quotient(total * c, ctas); }
  __device__ int of(int64_t x) const { return (int)quotient((x + 1) * ctas - 1, total); }
};

// A pair in the line of steps and a CTA's part of it.
struct Place {
  int row, hg, steps, here;   // here: its steps in this CTA
  int64_t begin, end;         // the first of them, and where the CTA's range ends
  bool whole, ends;           // whether its first step is here, and its last
};

// FULL: a warp for each of C::WARPS KV heads; all distances in shared memory are constants then.
template <typename T, int D, int NT, bool FULL>
__global__ void __launch_bounds__(32 * Cfg<T, D, NT>::WARPS, (Cfg<T, D, NT>::PER_SM))
kv4_decode_kernel(const __grid_constant__ Params p) {
  using C = Cfg<T, D, NT>;
  constexpr int NG = C::NG, RB = C::RB, QP = C::QP, PP = C::PP, U = C::U;
  extern __shared__ __align__(16) char smem[];
  __shared__ int64_t s_sum[C::WARPS];
  __shared__ int64_t s_before;
  __shared__ int s_row;
  // by step, four in turn: tokens that are not there; K and V have been copied; K has been read
  __shared__ __align__(16) uint8_t s_none[4][16 * C::WARPS * U];
  __shared__ uint64_t s_full[4], s_read[4];
  __shared__ Place s_place[C::WARPS][2];             // copied and read
  const auto& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int HG = FULL ? C::WARPS : p.HG, TS = FULL ? 1 : p.TS, warps = HG * TS;
  const int pitch = pitch_of(HG, RB);
  const int tokens = 16 * U * TS, half = tokens * pitch;   // of K or V of a step

  // ---- the CTA's range: a scan of all rows' steps
  const int each = (a.num_rows + (int)blockDim.x - 1) / (int)blockDim.x;
  const int r0 = min(a.num_rows, (int)threadIdx.x * each), r1 = min(a.num_rows, r0 + each);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += steps_of(p, a.seq_len[r], a.req_idx[r]);
  int64_t upto = mine;
#pragma unroll
  for (int x = 1; x < 32; x *= 2) {
    const int64_t y = __shfl_up_sync(~0u, upto, x);
    if (lane >= x) upto += y;
  }
  if (lane == 31) s_sum[warp] = upto;
  if (threadIdx.x < 4) {
    mbar_init(&s_full[threadIdx.x], 33 * warps);
    mbar_init(&s_read[threadIdx.x], warps);
    fence_mbar_init();
  }
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) upto += total;
    total += s_sum[w];
  }
  Cut cut;
  cut.total = total * p.groups;
  cut.ctas = (int)min((int64_t)gridDim.x, max((int64_t)1, cut.total));
  const bool idle = (int)blockIdx.x >= cut.ctas || total == 0;
  const int64_t begin = idle ? 0 : cut.begin(blockIdx.x);
  const int64_t end = idle ? 0 : cut.begin(blockIdx.x + 1);
  if (!idle) {
    const int64_t at = quotient(begin, p.groups);
    if (at >= upto - mine && at < upto) {
      int64_t before = upto - mine;
      int r = r0;
      for (; r + 1 < r1; ++r) {
        const int n = steps_of(p, a.seq_len[r], a.req_idx[r]);
        if (at < before + n) break;
        before += n;
      }
      s_row = r;
      s_before = before * p.groups;
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) p.w.range[blockIdx.x].row1 = -1;   // until a pair is begun and not ended
  // the first pair: the row's begun + 1st, of so many steps, the CTA's range beginning at that of them
  int first_steps = 1, begun = 0, first_step = 0;
  if (!idle) {
    first_steps = max(1, steps_of(p, a.seq_len[s_row], a.req_idx[s_row]));
    begun = (int)quotient(begin - s_before, first_steps);
    first_step = (int)(begin - s_before - (int64_t)begun * first_steps);
  }
  // what has to be written beside the pairs: rows without a token, and which CTAs share the first pair
  auto the_rest = [&] {
    if (warp == 0) {
      Range* rg = p.w.range + blockIdx.x;
      const int64_t at = begin - first_step;   // the pair's first step and, in odd lanes, its last
      const int cta = idle ? 0 : cut.of(lane & 1 ? at + first_steps - 1 : at);
      if (lane == 0) rg->row0 = first_step ? s_row : -1, rg->hg0 = begun, rg->start0 = cta;
      if (lane == 1) rg->last0 = cta;
    }
    for (int r = blockIdx.x; r < a.num_rows; r += gridDim.x) {
      const int len = a.seq_len[r];
      if (steps_of(p, len, a.req_idx[r])) continue;
      if (len != 0 && threadIdx.x == 0) set_status(p.status, kStatusPosRange);
      for (int x = threadIdx.x; x < a.num_q_heads * D; x += blockDim.x)
        ((T*)a.o)[(int64_t)r * a.num_q_heads * D + x] = Elem<T>::from_f(0.f);
      if (a.lse)
        for (int x = threadIdx.x; x < a.num_q_heads; x += blockDim.x)
          a.lse[(int64_t)r * a.num_q_heads + x] = -INFINITY;
    }
  };
  the_rest();
  if (idle) return;

  // ---- copies: K and V of step n, each into the next half of the ring, are issued when step n - 2 has
  // been read: the halves then held V of step n - 3 and K of step n - 2. Of the tokens a warp takes
  // 32 / HG at a time, HG lanes for each; with head counts that are no power of two some warps take as
  // many again
  const int rows_each = 32 / HG, piece = lane % HG;
  const int tok0 = warp * rows_each + lane / HG;   // the lane's first
  const bool copies = FULL || lane / HG < rows_each;
  const int further = warps * rows_each;           // from one of its tokens to the next
  constexpr int MOST = FULL ? U / 2 + U % 2 : U;   // tokens of a lane
  // Where a warp is in the line: what it needs when a pair ends is kept in shared memory, the steps left
  // of the pairs that are copied and read in registers
  Place& copied = s_place[warp][0];
  Place& at = s_place[warp][1];
  int copy_left, left;
  {
    Place x;
    x.row = s_row, x.hg = min(p.groups - 1, begun), x.steps = first_steps;
    x.begin = begin, x.end = end;
    x.here = (int)min((int64_t)(first_steps - first_step), end - begin);
    x.whole = first_step == 0, x.ends = first_step + x.here == first_steps;
    copy_left = left = x.here;
    if (lane == 0) copied = at = x;
    __syncwarp();
  }
  auto next_pair = [&](Place& place) {   // the steps of the next pair, 0: there is none
    Place x = place;
    x.begin += x.here;
    x.here = 0;
    if (x.begin < x.end) {
      if (++x.hg == p.groups) {
        x.hg = 0;
        do {
          ++x.row;
          x.steps = steps_of(p, a.seq_len[x.row], a.req_idx[x.row]);
        } while (x.steps == 0 && x.row + 1 < a.num_rows);
      }
      x.here = (int)min((int64_t)x.steps, x.end - x.begin);
      x.whole = true, x.ends = x.here == x.steps;
    }
    __syncwarp();
    if (lane == 0) place = x;
    __syncwarp();
    return x.here;
  };
  int column = 0;                    // of the lane's piece in a slot
  const int32_t* table = nullptr;    // the first token's slot
  int rest = 0;                      // tokens of the row from it on
  int slot[MOST];
  auto slots = [&] {
#pragma unroll
    for (int u = 0; u < MOST; ++u) slot[u] = rest > u * further ? table[u * further] : 0;
  };
  auto open_copies = [&](int step) {
    const int row = copied.row, pos = step * tokens + tok0;
    table = a.req_to_token + (int64_t)a.req_idx[row] * a.max_ctx + pos;
    rest = a.seq_len[row] - pos;
    column = copied.hg * HG * RB + piece * C::CH;
    slots();
  };
  const uint32_t full0 = smem_u32(&s_full[0]), read0 = smem_u32(&s_read[0]);
  auto next_half = [](int h, int by) { return h + by >= C::HALVES ? h + by - C::HALVES : h + by; };
  uint32_t to = 0;              // the step that is copied next
  int to_half = 0;              // where K goes
  const uint32_t dst0 = smem_u32(smem) + tok0 * pitch + piece * C::CH;
  const uint32_t none0 = smem_u32(&s_none[0][tok0]);
  const uint32_t slots_in = (uint32_t)min(a.num_slots, (int64_t)1 << 31);
  auto issue = [&] {
    const uint32_t kd = dst0 + to_half * half, vd = dst0 + next_half(to_half, 1) * half;
#pragma unroll
    for (int u = 0; u < MOST; ++u) {
      if (!(FULL && U % 2 == 0) && (!copies || tok0 + u * further >= tokens)) continue;
      const bool in = rest > u * further, good = in && (uint32_t)slot[u] < slots_in;
      if (in && !good) set_status(p.status, kStatusSlotRange);
      const int64_t from = (int64_t)(good ? slot[u] : 0) * p.stride + column;
      const char *ks = (const char*)a.k_pool + from, *vs = (const char*)a.v_pool + from;
#pragma unroll
      for (int i = 0; i < 5; ++i)
        cp_async_or_zero<C::CH>(kd + u * further * pitch + i * HG * C::CH, ks + i * HG * C::CH, good);
#pragma unroll
      for (int i = 0; i < 5; ++i)
        cp_async_or_zero<C::CH>(vd + u * further * pitch + i * HG * C::CH, vs + i * HG * C::CH, good);
      if (piece == 0)
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(none0 + (to & 3) * (16 * C::WARPS * U) + u * further),
                     "r"(good ? 0 : 1) : "memory");
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full0 + 8 * (to & 3))
                 : "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(&s_full[to & 3]);
    ++to;
    to_half = next_half(to_half, 2);
    if (--copy_left == 0) {
      copy_left = next_pair(copied);
      if (copy_left > 0) open_copies(0);
    } else {
      table += tokens, rest -= tokens;
      slots();
    }
  };

  // ---- the state of one pair: queries, maxima and sums, outputs
  const int hw = FULL ? warp : warp % HG, ts = FULL ? 0 : warp / HG;
  uint32_t qf[QP][NT][NG][2][2];   // query elements of the matrix steps of each group
  uint32_t qm[NT][3];              // sums of a group's query elements, in three bf16 parts
  float Q[C::F32 ? NT : 1][C::F32 ? NG : 1][2];   // the same in fp32, of heads 2t and 2t + 1
  float F[NT][2], mx[NT][2], l[NT][2];
  constexpr int NW = NG / 2;       // words of codes that a lane holds of a token's values
  float O[NT][NW][2][2][4];
  float M[NT][C::F32 ? 2 * NG : 4];
  auto begin_pair = [&] {
    const int row = at.row, h = at.hg * HG + hw;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qh = nt * 8 + g;
      float x[NG][8], most = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
#pragma unroll
        for (int n = 0; n < 8; ++n) x[j][n] = 0.f;
        if (qh < p.G) {
          const T* src = (const T*)a.q + ((int64_t)row * a.num_q_heads + h * p.G + qh) * D + 32 * j +
                         8 * t;
          if constexpr (C::F32) {
            const float4 u = ((const float4*)src)[0], v = ((const float4*)src)[1];
            x[j][0] = u.x, x[j][1] = u.y, x[j][2] = u.z, x[j][3] = u.w;
            x[j][4] = v.x, x[j][5] = v.y, x[j][6] = v.z, x[j][7] = v.w;
          } else {
            const uint4 u = *(const uint4*)src;
            x[j][0] = bf16lo(u.x), x[j][1] = bf16hi(u.x), x[j][2] = bf16lo(u.y), x[j][3] = bf16hi(u.y);
            x[j][4] = bf16lo(u.z), x[j][5] = bf16hi(u.z), x[j][6] = bf16lo(u.w), x[j][7] = bf16hi(u.w);
          }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) most = fmaxf(most, fabsf(x[j][n]));
      }
      most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
      most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
      // the head's elements over 2^e: below 2 in magnitude, exact. Scores are summed over 2^(e - UNIT) and
      // taken to base 2 by one factor: one too large for fp32 makes the scores NaN, one below 2^-118
      // goes with scores under 2^-80 (the first reference, the least number, is then still far below them)
      const int e = min(max((int)(__float_as_uint(most) >> 23) - 127, -126), 127);
      constexpr float unit = 1 << C::UNIT;
      const float f = a.sm_scale * __uint_as_float((uint32_t)(127 + e) << 23) * (kLog2e * unit);
      const float down = f > FLT_MAX ? __uint_as_float(0x7FC00000u)
                                     : __uint_as_float(e == 127 ? 1u << 22 : (uint32_t)(127 - e) << 23);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        float s = 0.f;
#pragma unroll
        for (int n = 0; n < 8; ++n) x[j][n] *= down, s += x[j][n];
        s += __shfl_xor_sync(~0u, s, 1);
        s += __shfl_xor_sync(~0u, s, 2);
        if (t == j) sum = s;
        if constexpr (C::F32)
#pragma unroll
          for (int k = 0; k < 2; ++k) Q[nt][j][k] = 0.25f * __shfl_sync(~0u, s, (2 * t + k) * 4);
        // a code's pattern is the bf16 number code * 2^-133 (or 16 times that), subnormal or next to
        // it, which times an element * 2^126 is code * element * 2^-7; fp32: (code - 8) * 2^-33 times
        // an element * 2^31
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float up = (C::F32 ? 0x1p31f : 0x1p126f) * (b ? 0.0625f : 1.f);
            float lo = x[j][2 * k + b] * up, hi = x[j][2 * k + b + 4] * up;
#pragma unroll
            for (int q = 0; q < QP; ++q) qf[q][nt][j][k][b] = take_part(lo, hi);
          }
      }
      float none = 0.f;
      sum /= unit;
#pragma unroll
      for (int k = 0; k < 3; ++k) qm[nt][k] = take_part(none, sum);
      const float factor = fminf(fmaxf(f, 0x1p-118f), FLT_MAX);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        F[nt][k] = __shfl_sync(~0u, factor, (2 * t + k) * 4);
        mx[nt][k] = -FLT_MAX, l[nt][k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < (C::F32 ? 2 * NG : 4); ++k) M[nt][k] = 0.f;
#pragma unroll
      for (int k = 0; k < 16 * NW; ++k) (&O[nt][0][0][0][0])[k] = 0.f;
    }
  };

  // scores of the warp's 16 tokens at kt: x[nt] = rows g, g + 8 x heads 2t, 2t + 1
  const int k_at = place<NG>(g) * pitch + 4 * NG * t;
  const int kp_at = place<NG>(g) * pitch + D / 2;
  const int eight = 8 * pitch;   // rows r and r + 8
  auto scores = [&](const char* kt, float (&x)[NT][4]) {
    uint32_t wa[NG], wb[NG], pa[NG], pb[NG];
    load(kt + k_at, wa);
    load(kt + k_at + eight, wb);
    load(kt + kp_at, pa);
    load(kt + kp_at + eight, pb);
    if constexpr (C::F32) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
    } else {
      uint32_t ma = 0, mb = 0;
      if (NG == 4 || t < NG) {
        ma = *(const uint32_t*)(kt + kp_at + 4 * t);
        mb = *(const uint32_t*)(kt + kp_at + 4 * t + eight);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_zero(x[nt], ma, mb, ma, mb, qm[nt][0], qm[nt][1]);
        mma(x[nt], ma, mb, ma, mb, qm[nt][2], 0);
      }
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      float d[NT][4], rest[NT][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t va = wa[j] >> 8 * k, vb = wb[j] >> 8 * k;
        uint32_t a0 = va & 0x000F000Fu, a1 = vb & 0x000F000Fu;
        uint32_t a2 = va & 0x00F000F0u, a3 = vb & 0x00F000F0u;
        if constexpr (C::F32) {   // (code - 8) * 2^-33, 16 times that: small sums lose less
          a0 = fma2(a0, pow2_bf16x2(100), kMinus | pow2_bf16x2(-30));
          a1 = fma2(a1, pow2_bf16x2(100), kMinus | pow2_bf16x2(-30));
          a2 = fma2(a2, pow2_bf16x2(100), kMinus | pow2_bf16x2(-26));
          a3 = fma2(a3, pow2_bf16x2(100), kMinus | pow2_bf16x2(-26));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const auto& q0 = qf[0][nt][j][k];
          if (k == 0)
            mma_zero(d[nt], a0, a1, a2, a3, q0[0], q0[1]);
          else
            mma(d[nt], a0, a1, a2, a3, q0[0], q0[1]);
          if constexpr (C::F32) {
            const auto& q1 = qf[1][nt][j][k];
            const auto& q2 = qf[2][nt][j][k];
            if (k == 0)
              mma_zero(rest[nt], a0, a1, a2, a3, q1[0], q1[1]);
            else
              mma(rest[nt], a0, a1, a2, a3, q1[0], q1[1]);
            mma(rest[nt], a0, a1, a2, a3, q2[0], q2[1]);
          }
        }
      }
      const float sa = bf16lo(pa[j]), sb = bf16lo(pb[j]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (C::F32) {
          const float ca = fmaf(8.f, sa, bf16hi(pa[j])), cb = fmaf(8.f, sb, bf16hi(pb[j]));
          x[nt][0] += fmaf(sa, d[nt][0], fmaf(sa, rest[nt][0], ca * Q[nt][j][0]));
          x[nt][1] += fmaf(sa, d[nt][1], fmaf(sa, rest[nt][1], ca * Q[nt][j][1]));
          x[nt][2] += fmaf(sb, d[nt][2], fmaf(sb, rest[nt][2], cb * Q[nt][j][0]));
          x[nt][3] += fmaf(sb, d[nt][3], fmaf(sb, rest[nt][3], cb * Q[nt][j][1]));
        } else {
          x[nt][0] = fmaf(sa, d[nt][0], x[nt][0]);
          x[nt][1] = fmaf(sa, d[nt][1], x[nt][1]);
          x[nt][2] = fmaf(sb, d[nt][2], x[nt][2]);
          x[nt][3] = fmaf(sb, d[nt][3], x[nt][3]);
        }
      }
    }
  };

  // outputs += weights x of the 16 tokens at vt times their values. A lane has 2 NW times four
  // elements, element(w, h) .., of tokens 2t, 2t + 1, 2t + 8, 2t + 9: all of group vj
  constexpr bool PAIRS = NG == 4;    // pairs of tokens come transposed from shared memory
  const int vj = g / (8 / NG), vt0 = g % (8 / NG) * NW;
  const int v_at = place<NG>(2 * t) * pitch + 4 * (vt0 * NG + vj);
  const int vp_at = place<NG>(2 * t) * pitch + D / 2 + 4 * vj;
  const int odd = (place<NG>(1) - place<NG>(0)) * pitch;   // rows 2t and 2t + 1
  const int row_at = place<NG>(lane & 15) * pitch + (lane >> 4) * 16;
  auto word = [](const char* at) { return *(const uint32_t*)at; };
  auto values = [&](const char* vt, float (&x)[NT][4]) {
    if constexpr (C::F32) {   // the groups' middles in fp32
      uint32_t pa[NG], pb[NG];
      load(vt + kp_at, pa);
      load(vt + kp_at + eight, pb);
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const float ca = fmaf(8.f, bf16lo(pa[j]), bf16hi(pa[j]));
        const float cb = fmaf(8.f, bf16lo(pb[j]), bf16hi(pb[j]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            M[nt][2 * j + c] += fmaf(x[nt][c], ca, x[nt][2 + c] * cb);
      }
    }
    uint32_t b[NT][PP][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < PP; ++k) {
        b[nt][k][0] = movmatrix_trans(take_part(x[nt][0], x[nt][1]));
        b[nt][k][1] = movmatrix_trans(take_part(x[nt][2], x[nt][3]));
      }
    uint32_t r01, r23, m01, m23;
    if constexpr (PAIRS) {   // column g of (scale, minimum) of all groups; the neighbour has the other
      ldmatrix_x2_trans(smem_u32(vt + row_at + D / 2 - (lane >> 4) * 16), m01, m23);
      const uint32_t o01 = __shfl_xor_sync(~0u, m01, 4), o23 = __shfl_xor_sync(~0u, m23, 4);
      r01 = g & 1 ? o01 : m01, r23 = g & 1 ? o23 : m23;
    } else {
      const uint32_t q0 = word(vt + vp_at), q1 = word(vt + vp_at + odd);
      const uint32_t q2 = word(vt + vp_at + eight), q3 = word(vt + vp_at + odd + eight);
      r01 = prmt(q0, q1, 0x5410), r23 = prmt(q2, q3, 0x5410);
      m01 = prmt(q0, q1, 0x7632), m23 = prmt(q2, q3, 0x7632);
    }
    const uint32_t s01 = mul2(r01, pow2_bf16x2(96)), s23 = mul2(r23, pow2_bf16x2(96));
    if constexpr (!C::F32) {
      // row g: weights times minima of the lane's group (with PAIRS in row g | 1); row g + 8: times scales
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float m[4];
        mma_zero(m, m01, r01, m23, r23, b[nt][PP - 1][0], b[nt][PP - 1][1]);
#pragma unroll
        for (int q = PP - 2; q >= 0; --q) mma(m, m01, r01, m23, r23, b[nt][q][0], b[nt][q][1]);
        add4(M[nt], m);
      }
    }
    // -8 times the scale, 16 times that
    const uint32_t e01 = mul2(s01, kMinus | pow2_bf16x2(-126)), e23 = mul2(s23, kMinus | pow2_bf16x2(-126));
    const uint32_t d01 = mul2(e01, pow2_bf16x2(-4)), d23 = mul2(e23, pow2_bf16x2(-4));
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      uint32_t pairs[4];   // of tokens 2t, 2t + 1 and of 2t + 8, 2t + 9: four elements, and four more
      if constexpr (PAIRS) {
        ldmatrix_x4_trans(smem_u32(vt + row_at) + 32 * w, pairs);
      } else {
        const char* at = vt + v_at + 4 * NG * w;
        const uint32_t w0 = word(at), w1 = word(at + odd), w2 = word(at + eight);
        const uint32_t w3 = word(at + odd + eight);
        pairs[0] = prmt(w0, w1, 0x5410), pairs[1] = prmt(w2, w3, 0x5410);
        pairs[2] = prmt(w0, w1, 0x7632), pairs[3] = prmt(w2, w3, 0x7632);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t v01 = pairs[2 * h], v23 = pairs[2 * h + 1];
        uint32_t v[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // code * 2^-133 (16 times that) times scale * 2^96, less 8 scales: eight bits, exact. Around
          // the groups' middles the sums stay small and lose less: with sums of code * scale, kept in the
          // matrix unit, 3.1 % of bf16 outputs were unlike those of 64 bits on a row of 131 071 tokens,
          // so 0.9 (326 and 338 us on 128 rows of 512 .. 8192 tokens, 32 + 32 heads); now 0.07
          const uint32_t va = v01 >> 8 * k, vb = v23 >> 8 * k;
          const uint32_t a0 = va & 0x000F000Fu, a1 = va & 0x00F000F0u;
          const uint32_t a2 = vb & 0x000F000Fu, a3 = vb & 0x00F000F0u;
          v[k][0] = fma2(a0, s01, d01), v[k][1] = fma2(a1, s01, e01);
          v[k][2] = fma2(a2, s23, d23), v[k][3] = fma2(a3, s23, e23);
        }
        // sums of 16 tokens from zero, the least parts first, and those added in fp32: a matrix instruction
        // cuts its sums off, always towards zero (kept there, sums of 32 000 positive values were 800 half
        // steps of fp32 too small, for 3 % less time)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            mma_zero(d[k], v[k][0], v[k][1], v[k][2], v[k][3], b[nt][PP - 1][0], b[nt][PP - 1][1]);
#pragma unroll
          for (int q = PP - 2; q >= 0; --q)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              mma(d[k], v[k][0], v[k][1], v[k][2], v[k][3], b[nt][q][0], b[nt][q][1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) add4(O[nt][w][h][k], d[k]);
        }
      }
    }
  };

  // the state of head 2t + c of tile nt: elements element(w, h) .. + 3
  auto element = [&](int w, int h) {
    return PAIRS ? 32 * vj + 8 * (2 * w + h) + 4 * (g & 1) : 32 * vj + 8 * (vt0 + w) + 4 * h;
  };
  auto outputs = [&](int nt, int c, int w, int h) {
    float m = M[nt][c];
    if constexpr (!C::F32) m = fmaf(8.f, M[nt][2 + c], PAIRS ? __shfl_sync(~0u, m, lane | 4) : m);
    if constexpr (C::F32)
#pragma unroll
      for (int j = 1; j < NG; ++j) m = vj == j ? M[nt][2 * j + c] : m;
    const auto& o = O[nt][w][h];
    return make_float4(fmaf(o[0][c], 0x1p37f, m), fmaf(o[0][2 + c], 0x1p33f, m),
                       fmaf(o[1][c], 0x1p37f, m), fmaf(o[1][2 + c], 0x1p33f, m));
  };
  // what a pair's head gave: the outputs, or a state in the workspace
  auto store = [&](int qh, int d, float4 v, float m, float den) {
    const int64_t head = (int64_t)at.row * a.num_q_heads + (at.hg * HG + hw) * p.G + qh;
    if (at.whole && at.ends) {
      const float f = den == 0.f ? 0.f : 1.f / den;
      T* o = (T*)a.o + head * D + d;
      if constexpr (C::F32)
        *(float4*)o = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
      else
        *(uint2*)o = make_uint2(pack2_bf16(v.x * f, v.y * f), pack2_bf16(v.z * f, v.w * f));
      if (a.lse && d == 0) a.lse[head] = den == 0.f ? -INFINITY : kLn2 * (m + log2f(den));
    } else {
      const int64_t i = (((int64_t)blockIdx.x * 2 + (at.whole ? 1 : 0)) * HG + hw) * p.G + qh;
      *(float4*)(p.w.o + i * D + d) = v;
      if (d == 0) *(float2*)(p.w.ml + i * 2) = make_float2(m, den);
    }
  };
  // The step that is read; negative from a wait on that gave up: the warp then goes through its steps without
  // waiting, copying or saying what it has read, and its pairs' sums, from this one on, are NaN. Others of
  // the CTA give up in turn, or have what they need: no output is made of what did not arrive.
  int now = 0;
  auto give_up = [&] { now |= INT_MIN, copy_left = 0; };
  auto end_pair = [&](char* stage) {
    if (now < 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) l[nt][0] = l[nt][1] = __int_as_float(0x7FC00000);
    }
    if (threadIdx.x == 0 && at.whole && !at.ends) {
      Range* rg = p.w.range + blockIdx.x;
      rg->row1 = at.row, rg->hg1 = at.hg, rg->last1 = cut.of(at.begin + at.steps - 1);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) mx[nt][c] = fmaxf(mx[nt][c] * F[nt][c], -FLT_MAX);   // to base 2
#pragma unroll
      for (int x = 4; x < 32; x *= 2) {
#pragma unroll
        for (int c = 0; c < 2; ++c) l[nt][c] += __shfl_xor_sync(~0u, l[nt][c], x);
        if constexpr (C::F32)
#pragma unroll
          for (int k = 0; k < 2 * NG; ++k) M[nt][k] += __shfl_xor_sync(~0u, M[nt][k], x);
      }
    }
    if (TS == 1) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int w = 0; w < 2 * NW; ++w) {
            const float4 v = outputs(nt, c, w >> 1, w & 1);
            const int qh = nt * 8 + 2 * t + c;
            if (qh < p.G) store(qh, element(w >> 1, w & 1), v, mx[nt][c], l[nt][c]);
          }
      return;
    }
    // warps that share a head join their states, a few heads at a time, in the half that all have read
    constexpr int H = U == 2 ? 4 : 2, STATE = H * (D + 2);
    float* own = (float*)stage + warp * STATE;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int part = 0; part < 8 / H; ++part) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int q8 = 2 * t + c, qh = q8 % H;
#pragma unroll
          for (int w = 0; w < 2 * NW; ++w) {
            const float4 v = outputs(nt, c, w >> 1, w & 1);
            if (q8 / H == part) *(float4*)(own + qh * D + element(w >> 1, w & 1)) = v;
          }
          if (g == 0 && q8 / H == part) own[H * D + qh] = mx[nt][c], own[H * D + H + qh] = l[nt][c];
        }
        __syncthreads();
        const int heads = min(H, p.G - nt * 8 - part * H);
        for (int x = ts * 32 + lane; x < heads * (D / 4); x += 32 * TS) {
          const int qh = x / (D / 4), d = x % (D / 4) * 4;
          float m = -FLT_MAX, den = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int s = 0; s < TS; ++s)
            m = fmaxf(m, ((const float*)stage)[(s * HG + hw) * STATE + H * D + qh]);
          for (int s = 0; s < TS; ++s) {
            const float* other = (const float*)stage + (s * HG + hw) * STATE;
            const float f = ex2(other[H * D + qh] - m);
            const float4 w = *(const float4*)(other + qh * D + d);
            den = fmaf(f, other[H * D + H + qh], den);
            v.x = fmaf(f, w.x, v.x), v.y = fmaf(f, w.y, v.y);
            v.z = fmaf(f, w.z, v.z), v.w = fmaf(f, w.w, v.w);
          }
          store(nt * 8 + part * H + qh, d, v, m, den);
        }
      }
  };

  open_copies(first_step);
  issue();
  if (copy_left > 0) issue();
  begin_pair();
  int now_half = 0;             // K of step `now`
  const int mine_at = ts * 16 * U * pitch + hw * RB;
  while (true) {
    if (now >= 0 && !wait_for(full0 + 8 * (now & 3), now >> 2 & 1, p)) give_up();
    float x[U][NT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) scores(smem + now_half * half + mine_at + u * 16 * pitch, x[u]);
    // tokens that are not there weigh nothing
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint8_t* gone = &s_none[now & 3][(ts * U + u) * 16];
      const uint4 none = *(const uint4*)gone;
      if (none.x | none.y | none.z | none.w) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (gone[place<NG>(g + 8 * k)])
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[u][nt][2 * k] = x[u][nt][2 * k + 1] = -INFINITY;
      }
    }
    __syncwarp();
    if (lane == 0 && now >= 0) mbar_arrive(&s_read[now & 3]);
    // the reference of a head's weights is a running maximum, as the scores are summed, that follows once
    // a weight is 2^8 and more. Differences are taken before the factor to base 2: against a product that
    // was rounded, scores of 2^30 and more lost their greatest weight or made it infinite
    bool beyond = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[nt][c] = fmaxf(x[0][nt][c], x[0][nt][2 + c]);
#pragma unroll
        for (int u = 1; u < U; ++u)
          top[nt][c] = fmaxf(top[nt][c], fmaxf(x[u][nt][c], x[u][nt][2 + c]));
        beyond |= (top[nt][c] - mx[nt][c]) * F[nt][c] > 8.f;
      }
    if (__any_sync(~0u, beyond)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int s = 4; s < 32; s *= 2)
            top[nt][c] = fmaxf(top[nt][c], __shfl_xor_sync(~0u, top[nt][c], s));
          const float to = fmaxf(mx[nt][c], top[nt][c]), f = ex2((mx[nt][c] - to) * F[nt][c]);
          mx[nt][c] = to;
          l[nt][c] *= f;
#pragma unroll
          for (int k = 0; k < (C::F32 ? NG : 2); ++k) M[nt][2 * k + c] *= f;
#pragma unroll
          for (int k = 0; k < 4 * NW; ++k) {
            float* o = &O[nt][0][0][0][0] + 4 * k + c;
            o[0] *= f, o[2] *= f;
          }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[u][nt][k] = ex2((x[u][nt][k] - mx[nt][k & 1]) * F[nt][k & 1]);
          l[nt][k & 1] += x[u][nt][k];
        }
    char* vt = smem + next_half(now_half, 1) * half;
#pragma unroll
    for (int u = 0; u < U; ++u) values(vt + mine_at + u * 16 * pitch, x[u]);
    if (--left == 0) end_pair(vt);
    __syncwarp();
    if (copy_left > 0) {
      if (wait_for(read0 + 8 * (now & 3), now >> 2 & 1, p))
        issue();
      else
        give_up();
    }
    ++now;
    now_half = next_half(now_half, 2);
    if (left > 0) continue;
    left = next_pair(at);
    if (left == 0) return;
    begin_pair();
  }
}

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;

// Joins the states of pairs that ranges cut. The CTAs that share a pair share its heads; few states: a
// warp for each head, many: all warps. Maxima, sums and the first eight outputs are asked for at once, the
// other outputs eight at a time (one row's 304 states of 64 heads: 16.8 us one by one, 10 so).
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads, 2) kv4_merge_kernel(const __grid_constant__ Params p) {
  __shared__ float so[kMergeWarps][D], sm[kMergeWarps], sl[kMergeWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int E = D / 32;
  const auto& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Range rg = p.w.range[blockIdx.x];
  const int heads = p.HG * p.G;
  for (int side = 0; side < 2; ++side) {
    const int row = side ? rg.row1 : rg.row0, hg = side ? rg.hg1 : rg.hg0;
    if (row < 0) continue;
    const int start = side ? (int)blockIdx.x : rg.start0, last = side ? rg.last1 : rg.last0;
    const int n = last - start + 1;
    const bool many = n > 16;
    const int team = many ? 1 : kMergeWarps, i0 = many ? warp : 0, di = many ? kMergeWarps : 1;
    const int mine = (n - i0 + di - 1) / di;   // states of this warp: i0, i0 + di, ..
    for (int h = (blockIdx.x - start) * team + (many ? 0 : warp); h < heads; h += n * team) {
      auto at = [&](int i) {
        const int c = i0 + i * di;
        return ((int64_t)(start + c) * 2 + (c == 0)) * heads + h;
      };
      // the first outputs are asked for with the maxima and sums
      float x0[8][E];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
#pragma unroll
        for (int e = 0; e < E; ++e) x0[u][e] = 0.f;
        if (u < mine) {
          const float* o = p.w.o + at(u) * D + lane * E;
          if constexpr (E == 4)
            *(float4*)x0[u] = *(const float4*)o;
          else
            *(float2*)x0[u] = *(const float2*)o;
        }
      }
      float2 ml[3];
      static_assert(kSms * (kMaxWarpsPerSm / 3) <= 8 * 32 * 3, "a lane has at most three of a warp's states");
      float m = -FLT_MAX;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int i = lane + 32 * k;
        ml[k] = i < mine ? *(const float2*)(p.w.ml + at(i) * 2) : make_float2(-FLT_MAX, 0.f);
        m = fmaxf(m, ml[k].x);
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
      if (many) {
        if (lane == 0) sm[warp] = m;
        __syncthreads();
        for (int w = 0; w < kMergeWarps; ++w) m = fmaxf(m, sm[w]);
      }
      float den = 0.f, f[3], v[E] = {};
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        f[k] = ex2(ml[k].x - m);
        den = fmaf(f[k], ml[k].y, den);
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) den += __shfl_xor_sync(~0u, den, x);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float fu = __shfl_sync(~0u, f[0], u);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf(fu, x0[u][e], v[e]);
      }
      for (int i = 8; i < mine; i += 8) {
        float x[8][E];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
#pragma unroll
          for (int e = 0; e < E; ++e) x[u][e] = 0.f;
          if (i + u < mine) {
            const float* o = p.w.o + at(i + u) * D + lane * E;
            if constexpr (E == 4)
              *(float4*)x[u] = *(const float4*)o;
            else
              *(float2*)x[u] = *(const float2*)o;
          }
        }
        const float fi = i < 32 ? f[0] : i < 64 ? f[1] : f[2];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float fu = __shfl_sync(~0u, fi, (i + u) & 31);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = fmaf(fu, x[u][e], v[e]);
        }
      }
      if (many) {
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane * E + e] = v[e];
        if (lane == 0) sl[warp] = den;
        __syncthreads();
        if (warp == 0) {
          den = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = 0.f;
#pragma unroll
          for (int w = 0; w < kMergeWarps; ++w) {
            den += sl[w];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] += so[w][lane * E + e];
          }
        }
        __syncthreads();
        if (warp != 0) continue;
      }
      const int64_t head = (int64_t)row * a.num_q_heads + (int64_t)hg * heads + h;
      const float by = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
      for (int e = 0; e < E; ++e)
        ((T*)a.o)[head * D + lane * E + e] = Elem<T>::from_f(v[e] * by);
      if (a.lse && lane == 0) a.lse[head] = den == 0.f ? -INFINITY : kLn2 * (m + log2f(den));
    }
  }
}

// ---------------------------------------------------------------- launches
// CTAs that may have a range, whatever the rows hold.
inline int64_t most_ctas(const Params& p) {
  const int64_t steps = (p.a.max_seq_len + p.tokens - 1) / p.tokens;
  const int64_t fit = kSms * std::max(1, kMaxWarpsPerSm / (p.HG * p.TS));
  return std::max<int64_t>(1, std::min<int64_t>(fit, steps * p.a.num_rows * p.groups));
}

template <typename T, int D, int NT>
int smem_of(int HG) {
  using C = Cfg<T, D, NT>;
  return C::HALVES * 16 * C::U * (C::WARPS / HG) * pitch_of(HG, C::RB);
}

struct Setup {
  int sms;
  int per_sm[9];   // CTAs, by KV heads of a CTA
};

template <typename T, int D, int NT>
cudaError_t launch_t(const Params& p, cudaStream_t s) {
  using C = Cfg<T, D, NT>;
  static PerDevice<Setup> setup;
  const Setup* st = nullptr;
  cudaError_t e = setup.get(
      [](Setup& x) {
        int dev = 0;
        cudaError_t r = cudaGetDevice(&dev);
        if (r == cudaSuccess)
          r = cudaDeviceGetAttribute(&x.sms, cudaDevAttrMultiProcessorCount, dev);
        for (int h = 1; h <= C::WARPS && r == cudaSuccess; ++h) {
          const auto kernel = h == C::WARPS ? kv4_decode_kernel<T, D, NT, true>
                                            : kv4_decode_kernel<T, D, NT, false>;
          r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
          if (r == cudaSuccess)
            r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                &x.per_sm[h], kernel, 32 * (C::WARPS / h * h), smem_of<T, D, NT>(h));
        }
        return r;
      },
      &st);
  if (e != cudaSuccess) return e;
  const int warps = p.HG * p.TS;
  const unsigned grid = (unsigned)std::min<int64_t>(
      most_ctas(p), (int64_t)st->sms * std::max(1, std::min(st->per_sm[p.HG], kMaxWarpsPerSm / warps)));
  const int smem = smem_of<T, D, NT>(p.HG);
  if (p.HG == C::WARPS)
    kv4_decode_kernel<T, D, NT, true><<<grid, 32 * warps, smem, s>>>(p);
  else
    kv4_decode_kernel<T, D, NT, false><<<grid, 32 * warps, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (grid == 1 || p.a.max_seq_len <= p.tokens) return cudaSuccess;   // no pair is cut
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_merge_kernel<T, D>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <typename T>
cudaError_t launch(const Params& p, cudaStream_t s) {
  if (p.a.head_dim == 128) return p.G <= 8 ? launch_t<T, 128, 1>(p, s) : launch_t<T, 128, 2>(p, s);
  return p.G <= 8 ? launch_t<T, 64, 1>(p, s) : launch_t<T, 64, 2>(p, s);
}
// Each type's kernels are compiled in a file of their own.
extern template cudaError_t launch<__nv_bfloat16>(const Params&, cudaStream_t);
extern template cudaError_t launch<float>(const Params&, cudaStream_t);

}  // namespace kv4
}  // namespace rc

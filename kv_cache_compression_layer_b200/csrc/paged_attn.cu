// kv_paged_attn: attention of a few query tokens per row over the paged 4-bit
// cache (formats in include/kvcomp_paged.h).
//
// What bounds it: the codes and scales are read once, d + 8 G bytes a token
// (144 at d = 128 and groups of 64), and 16 keys cost 370 instructions, 128 of
// them to unpack the codes. Neither is at its limit (DRAM at 0.4, issue and the
// logic pipe at 0.5): twelve attending warps an SM, each a chain of loads, unpacking,
// products, exponentials and products again, leave its latencies in the open. 192
// rows of 6400 keys (g = 8): 55.1 us, 3.2 TB/s (a form that let terms be cut at
// 2^-15 of the largest took 49). fp32: 77 us; 16 queries: 85; groups of 32: 65; d =
// 64: 35; one row of one key: 5.5 us.
//
// Products. With a group's step s and base m taken out of the sums,
//   q.k = sum_g s_g (q.c)_g + m_g (sum of q over g),
//   sum_j p_j v_j = sum_j p'_j c_j + sum_j p_j m_j,   p'_j = p_j s_j.
// Operands are 16-bit, sums float32. A pair of codes becomes 128 + c in two bf16
// with a shift and a logic instruction, c - 8 with one addition more (the bases
// then count m - 128 s or m + 8 s).
// Logits: bf16 queries are taken as they are times 128 + c, whose sums' last bits
// are 2^-23 of 143 sum |q| at most; with centred codes 192 rows of 6400 keys took
// 58.8 us against 54.8. fp32 queries are three bf16 each (24 bits) times c - 8.
// Outputs: p' is rounded to fp16 (2^-11 of a term) times c - 8 in fp16 (or-ed into
// 0x6400 a code is 1024 + c, into 0x5400 64 + c), under a scale, a power of two
// that a row's first keys choose. fp16 reaches from 2^-24 to 2^16, so this holds
// while steps stay within 2^10 of each other; before the first tile of which they
// do not (each lane looks at one key's), the row's sums drop the scale, and from
// there on p' is two bf16 (16 bits), which need none. So it is for a row's last
// keys too, and for fp32 with three bf16, always: no group, token or query costs
// another its bits. Two bf16 for all keys took 59.5 us, a scale for each query and
// group that follows its largest p' 60.5; rows that leave fp16 take 64.
// Both products have the cache as the 16-row operand (mma.sync m16n8k16: keys x
// queries, then channels x queries), so up to 8 queries cost no padding; a
// warp's fragments are one 16-byte load of K codes a key and 8-byte loads of V
// codes, free of bank conflicts by the page's order of words and the order in
// which a tile's keys take the rows.
//
// Work. Rows are cut into tiles of 128 tokens; a row costs its tiles plus a
// charge for starting and leaving it (an empty row 1). The CTAs (three an SM;
// two where 16 queries or fp32 take more registers) take equal shares of the
// total, contiguous over rows. In a CTA one warp runs ahead, over row ends too:
// it streams the tiles into a ring of stages with bulk copies (the four parts of
// a page are each contiguous) and lays out each row's queries as matrix
// fragments. Four warps take 16 tokens of each half of a tile, with a softmax
// of their own that is joined when the CTA leaves the row. CTAs that share a
// row leave partials: of each eight in turn the one that comes last, by a
// counter, joins them, and of those the last joins the eights (one CTA joining
// all of a row's took 37 us for four rows of 32768 keys, this takes 19; a
// kernel of its own for it cost every small call 4 us). Every sum has a fixed
// order.
#include <cuda_fp16.h>

#include <type_traits>

#include "paged_common.cuh"

namespace kvc {
namespace {

constexpr int kTile = 128;    // tokens per tile: two times 16 for each of the warps that attend
constexpr int kWarps = 4;     // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRowCost = 2;   // of starting and leaving a row, in tiles
constexpr int kMinShare = 2;  // cost of a CTA's share, at least
constexpr int kJoin = 8;      // partials joined at once
constexpr int kJoined = 1, kLost = 2;  // see last_of
// Steps times their scale that fp16 p' allow: weights are below 2^8, so p' stays below 2^15; the largest weight so far is 1
// or more, so its p' is 2^-3 or more, 2^22 times what rounding to the smallest fp16 takes from another.
constexpr float kReachLo = 0x1p-3f, kReachHi = 0x1p7f;
constexpr float kGrow = 8.f;  // the running maximum moves when a logit passes it by this (log2 units)

// Shared memory of a CTA: the ring of stages, the warps' outputs and (maximum,
// sum) on leaving a row, the rows' costs before them and lengths, two rows'
// queries (matrix fragments; per query its sums by group).
template <int D, int NG, int NT, bool F32>
struct Smem {
  static constexpr int kStages = D == 64 ? 4 : 2;  // as many as leave room for three CTAs an SM
  static constexpr int kCode = kTile * D / 2, kScale = kTile * NG * 4;
  static constexpr int kV = kCode, kKs = 2 * kCode, kVs = kKs + kScale, kStage = kVs + kScale;
  static constexpr int NQ = NT * 8, kORow = D + 4;
  static constexpr int kObuf = kStages * kStage;
  static constexpr int kMl = kObuf + kWarps * NQ * kORow * 4;
  static constexpr int kQ = kMl + kWarps * NQ * 8;
  static constexpr int kFrag = NQ * D * (F32 ? 6 : 2), kQBytes = kFrag + NQ * NG * 4;
  static constexpr int kBase = kQ + 2 * kQBytes;
  static constexpr int kLen = kBase + (kAttnRows + 1) * 4;
  static constexpr int kBar = (kLen + kAttnRows * 4 + 7) / 8 * 8;
  static constexpr int kBytes = kBar + (2 * kStages + 4) * 8 + 48;
};

// c += A B, A 16 x 16, B 16 x 8, both bf16, or (F16) fp16.
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two bf16 of a and b (lo in the low half), and what their rounding left of them.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ void rest2(uint32_t u, float& lo, float& hi) {
  lo -= lo_f(u);
  hi -= hi_f(u);
}
__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t add2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t add2_f16(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// The four nibble pairs of x (bits 4 n and 16 + 4 n) as two numbers c - 8 each, exactly: bf16, or (F16) fp16.
struct CodeConst {
  uint32_t k7, s7;            // bf16: 128, which a code or-ed into makes 128 + c, and -136, in both halves
  uint32_t k10, k6, s10, s6;  // fp16: 1024 and 64 (for a code in bits 4-7), -1032 and -72
};
template <bool F16, bool CENTRED = true>
__device__ __forceinline__ void codes8(uint32_t x, const CodeConst& k, uint32_t (&c)[4]) {
  if constexpr (F16) {
    const uint32_t y = x >> 8;
    c[0] = add2_f16(pick<0x000f000fu>(x, k.k10), k.s10);
    c[1] = add2_f16(pick<0x00f000f0u>(x, k.k6), k.s6);
    c[2] = add2_f16(pick<0x000f000fu>(y, k.k10), k.s10);
    c[3] = add2_f16(pick<0x00f000f0u>(y, k.k6), k.s6);
  } else {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      c[n] = pick<0x000f000fu>(x >> (4 * n), k.k7);
      if constexpr (CENTRED) c[n] = add2(c[n], k.s7);
    }
  }
}
struct AttnArgs {
  PageGeom g;
  SeqRows rows;
  PagedCache c;
  int row0, n_rows;  // call rows of this launch
  int n_q, group, R; // R = n_q * group
  float scale2, inv_scale2;  // log2(e) / sqrt(d)
  const void* q;
  void* out;
  float* lse;
  int* arrived;      // counters, 0 between calls: [chunks of queries][2 CTAs + kAttnRows] (see leave)
  float* part;
  unsigned long long limit_ns;
  CodeConst kc;  // an argument, so that the constants stay in registers
};

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// The NG scales of a token.
template <int NG>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&s)[NG]) {
  if constexpr (NG == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    s[0] = u.x, s[1] = u.y, s[2] = u.z, s[3] = u.w;
  } else if constexpr (NG == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    s[0] = u.x, s[1] = u.y;
  } else {
    s[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ int row_cost(int len) { return len > 0 ? (len + kTile - 1) / kTile + kRowCost : 1; }

// Equal shares of `cost` for n CTAs: CTA c has [lo(c), lo(c + 1)), lo(c) = floor(cost c / n).
struct Shares {
  int n, each, rest;
  __device__ __forceinline__ Shares(int cost, int grid) {
    n = max(1, min(grid, cost / kMinShare));
    each = cost / n;
    rest = cost - each * n;
  }
  __device__ __forceinline__ int lo(int c) const { return each * c + rest * c / n; }
  __device__ __forceinline__ int holder(int at) const {  // the CTA with lo(c) <= at < lo(c + 1)
    int c = min(n - 1, (int)__fdividef((float)at * (float)n, (float)each * (float)n + (float)rest));
    while (lo(c) > at) --c;
    while (c + 1 < n && lo(c + 1) <= at) ++c;
    return c;
  }
};

// The last of n rows with base[row] <= at, by the whole warp: 32 probes a round. base[0] = 0 <= at.
__device__ __forceinline__ int row_at(const int* base, int n, int at) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;  // in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const int i = lo + lane * step;
    const bool le = lane * step < len && base[i] <= at;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));
    len = min(step, len - last * step);
    lo += last * step;
  }
  return lo;
}

// The tiles [t0, t1) of a row of cost [b0, b1) that the CTA with costs [lo, hi) takes.
struct Share {
  int tiles, t0, t1;
};
__device__ __forceinline__ Share share_of(int b0, int b1, int lo, int hi) {
  Share s;
  s.tiles = max(0, b1 - b0 - kRowCost);
  s.t0 = max(lo - b0 - kRowCost, 0);
  s.t1 = min(s.tiles, hi - b0 - kRowCost);
  return s;
}

// The output of four channels of a query, o / L, in its type.
template <bool F32>
__device__ __forceinline__ void put4(void* out, long long at, float4 o, float L) {
  const float inv = L == 0.f ? 0.f : 1.f / L;
  if constexpr (F32)
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) =
        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
}
__device__ __forceinline__ float lse_of(float M, float L) {
  return L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <int D, int NG, int NT, bool F32>
__global__ void __launch_bounds__(kThreads, NT == 1 && !F32 ? kAttnCtasPerSm : 2) paged_attn_kernel(const AttnArgs a) {
  using S = Smem<D, NG, NT, F32>;
  constexpr int W = D / 32, NQ = S::NQ, QP = F32 ? 3 : 1, kChain = F32 ? 8 : 32, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  float* obuf = reinterpret_cast<float*>(smem + S::kObuf);
  float2* ml = reinterpret_cast<float2*>(smem + S::kMl);
  int* base = reinterpret_cast<int*>(smem + S::kBase);
  int* lens = reinterpret_cast<int*>(smem + S::kLen);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;  // [2], by the parity of the row's number in this CTA
  uint64_t* q_empty = q_full + 2;
  int* wsum = reinterpret_cast<int*>(q_empty + 2);  // [5]
  int* abort_flag = wsum + 10;
  int* last_flag = wsum + 11;
  const PageGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], kWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  // base[i]: cost of the rows before row i; every thread sums a run of rows
  {
    const int per = (a.n_rows + kThreads - 1) / kThreads;
    const int i0 = threadIdx.x * per, i1 = min(a.n_rows, i0 + per);
    int sum = 0;
    for (int i = i0; i < i1; ++i) {
      int n = a.c.len[table_row(a.rows, a.row0 + i)];
      if (n < 0 || n > (g.max_pages << g.log_p)) {
        n = 0;
        if (blockIdx.x == 0) atomicOr(a.c.status, KV_DEV_BOUNDS);
      }
      lens[i] = n;
      base[i] = sum;  // made absolute below
      sum += row_cost(n);
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int i = 0; i < warp; ++i) before += wsum[i];
    for (int i = i0; i < i1; ++i) base[i] += before;
    if (i1 == a.n_rows && i0 < a.n_rows) base[a.n_rows] = before + sum;
    __syncthreads();
  }
  const Shares shares(base[a.n_rows], gridDim.x);
  const int cta = blockIdx.x, chunk = blockIdx.y;  // the chunk of NQ query rows
  if (cta >= shares.n) return;
  const int lo = shares.lo(cta), hi = shares.lo(cta + 1);
  const int row = row_at(base, a.n_rows, lo);
  const Guard guard{abort_flag, a.c.status, a.limit_ns};
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return (bool)__all_sync(0xffffffffu, wait_bounded(bar, parity, guard));
  };
  const int grp = lane >> 2, tig = lane & 3;
  const int q0 = chunk * NQ, nq = min(NQ, a.R - q0);

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    const int part_tokens = min(g.P, kTile), ppt = kTile / part_tokens;  // pages per tile
    const int pg = lane >> 2, sec = lane & 3;
    const bool mine = pg < ppt;
    const uint32_t sec_bytes = sec < 2 ? part_tokens * (D / 2) : part_tokens * NG * 4;
    const int sec_page = sec == 0 ? 0 : sec == 1 ? g.v : sec == 2 ? g.ks : g.vs;
    const int sec_stage = sec == 0 ? 0 : sec == 1 ? S::kV : sec == 2 ? S::kKs : S::kVs;
    const uint32_t tok_bytes = sec < 2 ? D / 2 : NG * 4;
    int it = 0, st = 0, k = 0;  // tiles and rows so far; the stage that is next
    uint32_t turn = 0;          // the ring's turns, odd or even
    bool ok = true;
    for (int r = row; ok && r < a.n_rows && base[r] < hi; ++r) {
      const Share sh = share_of(base[r], base[r + 1], lo, hi);
      if (sh.t0 >= sh.t1) continue;
      const int32_t* list = a.c.table + (size_t)table_row(a.rows, a.row0 + r) * g.max_pages;
      const int np = (lens[r] + g.P - 1) >> g.log_p;
      int win = (sh.t0 * kTile) >> g.log_p;  // lane l holds page number list[win + l]
      int entry = win + lane < np ? list[win + lane] : -1;
      for (int t = sh.t0; t < sh.t1; ++t, ++it) {
        const int j0 = (t * kTile) >> g.log_p;
        if (j0 + ppt > win + 32) {
          win = j0;
          entry = win + lane < np ? list[win + lane] : -1;
        }
        const int page = __shfl_sync(0xffffffffu, entry, min(31, j0 - win + pg));
        const bool there = mine && j0 + pg < np;
        const bool good = there && page >= 0 && page < g.n_pages;
        if (there && !good) atomicOr(a.c.status, KV_DEV_BOUNDS);
        if (it >= kStages) ok = wait(&empty[st], (turn & 1) ^ 1);
        if (!ok) break;
        const unsigned n_good = __popc(__ballot_sync(0xffffffffu, good && sec == 0));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], n_good * part_tokens * (D + 8 * NG));
        __syncwarp();
        if (good) {
          const uint8_t* src =
              a.c.pages + (size_t)page * g.bytes + sec_page + ((t * kTile) & (g.P - 1)) * tok_bytes;
          bulk_load(smem + st * S::kStage + sec_stage + pg * part_tokens * tok_bytes, src, sec_bytes, &full[st]);
        }
        if (++st == kStages) {
          st = 0;
          ++turn;
        }
        if (t > sh.t0) continue;
        // with the row's first tile under way, its queries
        if (k >= 2) ok = wait(&q_empty[k & 1], ((k >> 1) - 1) & 1);
        if (!ok) {
          ++it;  // this tile's copy is under way
          break;
        }
        // as fragments, with their sums by group
        {
          uint4* frag = reinterpret_cast<uint4*>(smem + S::kQ + (k & 1) * S::kQBytes);
          float* meta = reinterpret_cast<float*>(smem + S::kQ + (k & 1) * S::kQBytes + S::kFrag);
  #pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int qi = nt * 8 + grp;
            float x[W][8], sum[NG];
  #pragma unroll
            for (int w = 0; w < W; ++w) {
              const long long at = ((long long)(a.row0 + r) * a.R + q0 + qi) * D + 32 * w + 8 * tig;
              if (qi < nq) {
                if (F32) {
                  const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
                  const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + 4);
                  x[w][0] = u.x, x[w][1] = u.y, x[w][2] = u.z, x[w][3] = u.w;
                  x[w][4] = v.x, x[w][5] = v.y, x[w][6] = v.z, x[w][7] = v.w;
                } else {
                  const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at);
                  x[w][0] = lo_f(u.x), x[w][1] = hi_f(u.x), x[w][2] = lo_f(u.y), x[w][3] = hi_f(u.y);
                  x[w][4] = lo_f(u.z), x[w][5] = hi_f(u.z), x[w][6] = lo_f(u.w), x[w][7] = hi_f(u.w);
                }
              } else {
  #pragma unroll
                for (int n = 0; n < 8; ++n) x[w][n] = 0.f;
              }
            }
  #pragma unroll
            for (int z = 0; z < NG; ++z) sum[z] = 0.f;
  #pragma unroll
            for (int w = 0; w < W; ++w) {
  #pragma unroll
              for (int n = 0; n < 8; ++n) sum[w * NG / W] += x[w][n];
  #pragma unroll
              for (int p = 0; p < QP; ++p) {
                uint32_t f[4];  // a code pair holds channels n and n + 4
  #pragma unroll
                for (int n = 0; n < 4; ++n) {
                  f[n] = pack2(x[w][n], x[w][n + 4]);
                  rest2(f[n], x[w][n], x[w][n + 4]);
                }
                frag[((nt * QP + p) * W + w) * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
              }
            }
  #pragma unroll
            for (int z = 0; z < NG; ++z) {
              sum[z] += __shfl_xor_sync(0xffffffffu, sum[z], 1);
              sum[z] += __shfl_xor_sync(0xffffffffu, sum[z], 2);
              if (tig == 0) meta[qi * NG + z] = sum[z];
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[k & 1]);
          ++k;
        }
      }
    }
    // copies in flight land before the CTA gives its memory back, also when the others have given up
    for (int i = max(0, it - kStages); i < it; ++i) wait_drain(&full[i % kStages], (i / kStages) & 1);
    return;
  }

  // -------------------------------------------------------------- consumers
  const CodeConst kc = a.kc;
  // Matrix row r of a half tile is token tok(r): rows 2 t and 2 t + 1 are tokens t and 4 + (t ^ 1), so that the
  // lanes of a K load and of a V load fall on different banks.
  const int krow = warp * 16 + ((grp & 1) ? 4 + ((grp >> 1) ^ 1) : grp >> 1);
  const int vrow = warp * 16 + tig, vrow2 = warp * 16 + 4 + (tig ^ 1);
  const int vplace = grp ^ ((tig & 2) << 1);
  int st = 0, k = 0;  // the stage that is next, rows so far
  uint32_t turn = 0;
  bool ok = true;
  for (int r = row; r < a.n_rows && base[r] < hi; ++r) {
    const Share sh = share_of(base[r], base[r + 1], lo, hi);
    const int crow = a.row0 + r;
    const bool whole = sh.t0 == 0 && sh.t1 == sh.tiles;
    if (sh.t0 >= sh.t1) {
      if (sh.tiles == 0) {  // an empty row
        const long long at = (long long)crow * a.R + q0;
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + at * (D * (F32 ? 4 : 2)));
        for (int i = threadIdx.x; i < nq * D * (F32 ? 4 : 2) / 16; i += kWarps * 32) o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse && (int)threadIdx.x < nq) a.lse[at + threadIdx.x] = -INFINITY;
      }
      continue;
    }
    const int len = lens[r];
    // CTAs that share the row (the first and the last hold its first and last tile)
    const int c_first = whole ? cta : shares.holder(base[r] + kRowCost);
    const int c_count = whole ? 1 : shares.holder(base[r + 1] - 1) - c_first + 1;
    // Counts this CTA's partial of a shared row. The row's CTAs come in eights; `first`, the slot of an eight's first
    // partial, has the eight's counter, the row counts the eights that are complete. 0 but for the last of n, for which
    // it is kJoined, or kLost where one had `lost` its partial (counted in the upper half): then nothing is joined.
    int* arrived = a.arrived + chunk * (2 * gridDim.x + kAttnRows);
    auto last_of = [&](int* counter, int n, bool lost) {
      const int add = lost ? 0x10001 : 1, now = atomicAdd(counter, add) + add;
      if ((now & 0xffff) != n) return 0;
      *counter = 0;
      return now > 0xffff ? kLost : kJoined;
    };
    const int c_own = cta - c_first, eight = c_own / kJoin;
    const int eights = (c_count + kJoin - 1) / kJoin, in_eight = min(kJoin, c_count - eight * kJoin);
    const int first = eight == 0 ? 2 * c_first + 1 : 2 * (c_first + eight * kJoin);
    auto give_up_row = [&] {  // a wait ran out: the row's counters stay in step all the same
      if (!whole && threadIdx.x == 0 && last_of(arrived + first, in_eight, true) && eights > 1)
        last_of(arrived + 2 * gridDim.x + r, eights, true);
    };
    if (!ok) {
      give_up_row();
      continue;
    }
    ok = wait(&q_full[k & 1], (k >> 1) & 1);

    // query fragments and their sums by group
    uint32_t qf[NT][QP][W][4];
    float qsum[NT][NG][2];
    {  // (where the wait ran out, of what lies there: it meets no key, and the row's output stays)
      const uint4* frag = reinterpret_cast<const uint4*>(smem + S::kQ + (k & 1) * S::kQBytes);
      const float* meta = reinterpret_cast<const float*>(smem + S::kQ + (k & 1) * S::kQBytes + S::kFrag);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int p = 0; p < QP; ++p)
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const uint4 u = frag[((nt * QP + p) * W + w) * 32 + lane];
            qf[nt][p][w][0] = u.x, qf[nt][p][w][1] = u.y, qf[nt][p][w][2] = u.z, qf[nt][p][w][3] = u.w;
          }
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // this lane's columns are queries 2 tig + c
          const float* mq = meta + (nt * 8 + 2 * tig + c) * NG;
#pragma unroll
          for (int z = 0; z < NG; ++z) qsum[nt][z][c] = mq[z];
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_empty[k & 1]);
    ++k;
    // keys that this lane's queries see
    int lim[NT][2];
    const int lim_min = len - a.n_q + 1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int qi = nt * 8 + 2 * tig + x;
        lim[nt][x] = qi < nq ? lim_min + (q0 + qi) / a.group : len;
      }

    float O[NT][2 * W][4], off[NT][NG][2], m2[NT][2], thr[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < NG; ++x) off[nt][x][0] = off[nt][x][1] = 0.f;
      m2[nt][0] = m2[nt][1] = thr[nt][0] = thr[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    float om = F32 ? 1.f : 0.f;  // the scale of p' and O; 0: not yet chosen
    bool wide = F32;             // no scale any more: steps lay too far apart
    bool moved = false;          // sums lie in the warp's part of obuf
    // This lane's four channels of part h of a row and query (nt, x) there.
    auto spot = [&](int nt, int x, int h) {
      return reinterpret_cast<float4*>(obuf + (warp * NQ + nt * 8 + 2 * tig + x) * S::kORow + 32 * h + 4 * grp);
    };


    // The warp's 16 keys of each of the halves u0 .. u0 + U - 1 of tile t in stage st; MASKED: some may be hidden from
    // some query, and steps may lie apart (WIDE). False: not done, since they do.
    auto attend = [&](auto uu, auto mk, const uint8_t* st, int u0, int t) {
      constexpr int U = decltype(uu)::value;
      constexpr bool MASKED = decltype(mk)::value, WIDE = MASKED || F32;
      constexpr int PP = F32 ? 3 : WIDE ? 2 : 1;
      const int row0 = krow + 64 * u0;          // token of the tile in matrix row grp; row grp + 8 is 8 further
      const int key0 = t * kTile + row0;
      // ---- logits: rows keys, columns queries
      float y[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t kw[2][W], ks[2][NG];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t* kp = st + (row0 + 64 * u + 8 * x) * (D / 2) + tig * (D / 8);
          if constexpr (W == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(kp);
            kw[x][0] = v.x, kw[x][1] = v.y, kw[x][2] = v.z, kw[x][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(kp);
            kw[x][0] = v.x, kw[x][1] = v.y;
          }
          load_scales<NG>(st + S::kKs + (row0 + 64 * u + 8 * x) * (NG * 4), ks[x]);
        }
        float acc[NT][NG][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < NG; ++x)
#pragma unroll
            for (int z = 0; z < 4; ++z) acc[nt][x][z] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t c0[4], c1[4];
          codes8<false, F32>(kw[0][w], kc, c0);
          codes8<false, F32>(kw[1][w], kc, c1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = QP - 1; p >= 0; --p) {
              mma<false>(acc[nt][w * NG / W], c0[0], c1[0], c0[1], c1[1], qf[nt][p][w][0], qf[nt][p][w][1]);
              mma<false>(acc[nt][w * NG / W], c0[2], c1[2], c0[3], c1[3], qf[nt][p][w][2], qf[nt][p][w][3]);
            }
        }
#pragma unroll
        for (int x = 0; x < NG; ++x)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float sc = lo_f(ks[z][x]), ad = fmaf(F32 ? 8.f : -128.f, sc, hi_f(ks[z][x]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float add = x == 0 ? ad * qsum[nt][x][c] : fmaf(ad, qsum[nt][x][c], y[u][nt][2 * z + c]);
                y[u][nt][2 * z + c] = fmaf(sc, acc[nt][x][2 * z + c], add);
              }
          }
        if constexpr (MASKED) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (key0 + 8 * (x >> 1) >= lim[nt][x & 1]) y[u][nt][x] = -INFINITY;
        }
      }
      uint32_t vs[U][2][NG];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          load_scales<NG>(st + S::kVs + (row0 + 64 * u + 8 * x) * (NG * 4), vs[u][x]);
          if constexpr (MASKED) {
            if (key0 + 8 * x >= len) {
#pragma unroll
              for (int z = 0; z < NG; ++z) vs[u][x][z] = 0;  // what lies there may be NaN
            }
          }
        }
      // ---- softmax: the running maximum follows only when a logit passes it by far
      bool grow = false, odd = false;
      if constexpr (!F32) {
        if (!wide && u0 == 0) {  // the steps of the warp's 32 keys of the tile, a key a lane
          const int at = warp * 16 + (lane & 15) + 64 * (lane >> 4);
          uint32_t sw[NG];
          load_scales<NG>(st + S::kVs + at * (NG * 4), sw);
#pragma unroll
          for (int z = 0; z < NG; ++z) {
            const float x = lo_f(sw[z]) * om;
            odd |= !(x >= kReachLo && x <= kReachHi);
          }
          if (MASKED) odd &= t * kTile + at < len;
          grow = odd;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) grow |= y[u][nt][x] > thr[nt][x & 1];
      if (__any_sync(0xffffffffu, grow)) {
        if constexpr (!F32) {
          if (__any_sync(0xffffffffu, odd)) {
            // the row's first keys choose the scale; steps that are out of its reach end it
            float top = 0.f, low = INFINITY;
            const int at = warp * 16 + (lane & 15) + 64 * (lane >> 4);
            if (t * kTile + at < len) {
              uint32_t sw[NG];
              load_scales<NG>(st + S::kVs + at * (NG * 4), sw);
#pragma unroll
              for (int z = 0; z < NG; ++z) {
                const float sc = lo_f(sw[z]);
                top = fmaxf(top, sc);
                low = sc >= 0.f ? fminf(low, sc) : 0.f;  // NaN: out of reach
              }
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
            }
            const bool first = om == 0.f;
            if (first) om = pow2(4 - min(100, max(-96, (int)(__float_as_uint(top) >> 23) - 127)));
            if (!first || !(top * om <= kReachHi && low * om >= kReachLo)) {
              wide = true;
              const float inv = __frcp_rn(om);
              om = 1.f;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2 * W; ++h)
#pragma unroll
                  for (int x = 0; x < 4; ++x) O[nt][h][x] *= inv;
              if (!WIDE) return false;
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float mx = fmaxf(y[0][nt][x], y[0][nt][2 + x]);
            if constexpr (U == 2) mx = fmaxf(mx, fmaxf(y[1][nt][x], y[1][nt][2 + x]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float now = fmaxf(m2[nt][x], mx * a.scale2);
            const float f = now == m2[nt][x] ? 1.f : ex2_approx(m2[nt][x] - now);
            m2[nt][x] = now;
            thr[nt][x] = (now + kGrow) * a.inv_scale2;
            l[nt][x] *= f;
#pragma unroll
            for (int z = 0; z < NG; ++z) off[nt][z][x] *= f;
#pragma unroll
            for (int z = 0; z < 2 * W; ++z) {
              O[nt][z][x] *= f;
              O[nt][z][2 + x] *= f;
            }
            if (moved) {
#pragma unroll
              for (int h = 0; h < W; ++h) {
                const float4 v = *spot(nt, x, h);
                *spot(nt, x, h) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
              }
            }
          }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t b[NT][NG][PP][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4], po[4];
          bool seen[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            seen[x] = !MASKED || key0 + 8 * (x >> 1) < lim[nt][x & 1];
            p[x] = ex2_approx(fmaf(y[u][nt][x], a.scale2, -m2[nt][x & 1]));
            if (!seen[x]) p[x] = 0.f;
            l[nt][x & 1] += p[x];
            po[x] = F32 ? p[x] : p[x] * om;
          }
#pragma unroll
          for (int z = 0; z < NG; ++z) {
            float ps[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float sc = lo_f(vs[u][x >> 1][z]), ba = fmaf(8.f, sc, hi_f(vs[u][x >> 1][z]));
              ps[x] = po[x] * sc;
              if constexpr (MASKED) {
                off[nt][z][x & 1] += seen[x] ? p[x] * ba : 0.f;  // a token that another query sees may be NaN
                if (!seen[x]) ps[x] = 0.f;
              } else {
                off[nt][z][x & 1] = fmaf(p[x], ba, off[nt][z][x & 1]);
              }
            }
#pragma unroll
            for (int part = 0; part < PP; ++part) {
              const uint32_t u0 = WIDE ? pack2(ps[0], ps[1]) : pack2_f16(ps[0], ps[1]);
              const uint32_t u1 = WIDE ? pack2(ps[2], ps[3]) : pack2_f16(ps[2], ps[3]);
              b[nt][z][part][0] = transpose8(u0);
              b[nt][z][part][1] = transpose8(u1);
              rest2(u0, ps[0], ps[1]);
              rest2(u1, ps[2], ps[3]);
            }
          }
        }
        // ---- output: rows channels, columns queries
        uint32_t vw[4][(W + 1) / 2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int vr = ((x & 1) ? vrow2 : vrow) + (x >> 1) * 8 + 64 * (u0 + u);
          const uint8_t* vp = st + S::kV + vr * (D / 2) + vplace * (D / 16);
          if constexpr (W == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(vp);
            vw[x][0] = v.x, vw[x][1] = v.y;
          } else {
            vw[x][0] = *reinterpret_cast<const uint32_t*>(vp);
          }
        }
#pragma unroll
        for (int h = 0; h < W; ++h) {
          const uint32_t sel = (h & 1) ? 0x7632u : 0x5410u;
          const uint32_t xx = __byte_perm(vw[0][h >> 1], vw[1][h >> 1], sel);
          const uint32_t yy = __byte_perm(vw[2][h >> 1], vw[3][h >> 1], sel);
          uint32_t c0[4], c1[4];
          codes8<!WIDE>(xx, kc, c0);
          codes8<!WIDE>(yy, kc, c1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = PP - 1; p >= 0; --p) {
              const uint32_t b0 = b[nt][h * NG / W][p][0], b1 = b[nt][h * NG / W][p][1];
              mma<!WIDE>(O[nt][2 * h], c0[0], c0[1], c1[0], c1[1], b0, b1);
              mma<!WIDE>(O[nt][2 * h + 1], c0[2], c0[3], c1[2], c1[3], b0, b1);
            }
        }
      }
      return true;
    };

    // The matrix unit cuts a running sum's last bits off, towards zero, at each of two products a tile (fp32: six):
    // after kChain tiles the sums go to the warp's place in shared memory, where additions round to nearest.
    for (int t = sh.t0; ok && t < sh.t1;) {
      const int end = min(sh.t1, t + kChain);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2 * W; ++x)
#pragma unroll
          for (int z = 0; z < 4; ++z) O[nt][x][z] = 0.f;
      for (; t < end; ++t) {
        ok = wait(&full[st], turn & 1);
        if (!ok) break;
        const uint8_t* stage = smem + st * S::kStage;
        const int tok = t * kTile + warp * 16;
        // both halves at once where every query sees all of them and the registers allow (16 queries spill, 192 rows of
        // 6400 keys, g = 16, 82 us against 74 when measured; 8 queries with groups of 32, 60.7 against 58; 8 with groups
        // of 64, 49.8 against 53.5 one after the other)
        constexpr int U = NT == 1 && (NG < 4 || F32) ? 2 : 1;
        bool done = false;
        if (tok + 64 + 16 <= lim_min && (F32 || !wide)) {
          done = attend(std::integral_constant<int, U>{}, std::false_type{}, stage, 0, t);
          if (U == 1 && done) attend(std::integral_constant<int, U>{}, std::false_type{}, stage, 1, t);
        }
        if (!done) {
#pragma unroll 1
          for (int u = 0; u < 2 && tok + 64 * u < len; ++u)
            attend(std::integral_constant<int, 1>{}, std::true_type{}, stage, u, t);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (++st == kStages) {
          st = 0;
          ++turn;
        }
      }
      const float inv = om > 0.f ? __frcp_rn(om) : 0.f;  // 0: the warp had no key
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int h = 0; h < W; ++h) {
            float4 v = moved ? *spot(nt, x, h) : make_float4(0.f, 0.f, 0.f, 0.f);
            v.x = fmaf(O[nt][2 * h][x], inv, v.x);
            v.y = fmaf(O[nt][2 * h][2 + x], inv, v.y);
            v.z = fmaf(O[nt][2 * h + 1][x], inv, v.z);
            v.w = fmaf(O[nt][2 * h + 1][2 + x], inv, v.w);
            *spot(nt, x, h) = v;
          }
      moved = true;
    }

    // ---- the CTA leaves the row: the warps' sums are joined
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], o);
        const int qi = nt * 8 + 2 * tig + x;
#pragma unroll
        for (int z = 0; z < NG; ++z) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) off[nt][z][x] += __shfl_xor_sync(0xffffffffu, off[nt][z][x], o);
        }
#pragma unroll
        for (int h = 0; h < W; ++h) {
          const float add = off[nt][h * NG / W][x];
          const float4 v = *spot(nt, x, h);
          *spot(nt, x, h) = make_float4(v.x + add, v.y + add, v.z + add, v.w + add);
        }
        if (grp == 0) ml[warp * NQ + qi] = make_float2(m2[nt][x], l[nt][x]);
      }
    }
    ok = named_bar_and(1, kWarps * 32, ok);
    if (!ok) {
      give_up_row();
      continue;
    }
    constexpr size_t kPart = kAttnQ * (D + 2);  // floats: (max, sum) and the output of up to kAttnQ query rows
    float* parts = a.part + (size_t)chunk * gridDim.x * 2 * kPart;
    float* part = parts + (size_t)(cta * 2 + (c_own == 0 ? 1 : 0)) * kPart;
    for (int i = threadIdx.x; i < nq * (D / 4); i += kWarps * 32) {
      const int qi = i / (D / 4), dim = 4 * (i - qi * (D / 4));
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * NQ + qi].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 e = ml[w * NQ + qi];
        const float f = e.x == M ? 1.f : ex2_approx(e.x - M);
        const float4 v = *reinterpret_cast<const float4*>(obuf + (w * NQ + qi) * S::kORow + dim);
        L += e.y * f;
        o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
      }
      if (whole) {
        const long long at = (long long)crow * a.R + q0 + qi;
        put4<F32>(a.out, at * D + dim, o, L);
        if (a.lse && dim == 0) a.lse[at] = lse_of(M, L);
      } else {
        *reinterpret_cast<float4*>(part + 2 * kAttnQ + qi * D + dim) = o;
        if (dim == 0) reinterpret_cast<float2*>(part)[qi] = make_float2(M, L);
      }
    }
    if (whole) {
      named_bar_sync(1, kWarps * 32);  // the buffer is free again
      continue;
    }
    // a shared row: joins n partials, the first at slot s0 and the others at slots s1, s1 + ds, ..
    auto join = [&](int n, int s0, int s1, int ds, bool last) {
      const int items = nq * (D / 4);
      for (int i0 = threadIdx.x; i0 < items; i0 += 2 * kWarps * 32) {  // two items' loads at once
        float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f};
        float4 o[2];
        o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int qi[2] = {i0 / (D / 4), min(i0 + kWarps * 32, items - 1) / (D / 4)};
        const int dim = 4 * (i0 % (D / 4));  // of both: the threads are a multiple of D / 4
        for (int c = 0; c < n; c += kJoin) {
          float2 e[2][kJoin];
          float4 v[2][kJoin];
#pragma unroll
          for (int x = 0; x < kJoin; ++x) {
            const int at = min(c + x, n - 1);
            const float* p = parts + (size_t)(at == 0 ? s0 : s1 + (at - 1) * ds) * kPart;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              e[y][x] = __ldcg(reinterpret_cast<const float2*>(p) + qi[y]);
              v[y][x] = __ldcg(reinterpret_cast<const float4*>(p + 2 * kAttnQ + qi[y] * D + dim));
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float m = M[y];
#pragma unroll
            for (int x = 0; x < kJoin; ++x) m = fmaxf(m, e[y][x].x);
            const float f0 = M[y] == m ? 1.f : ex2_approx(M[y] - m);
            L[y] *= f0;
            o[y].x *= f0, o[y].y *= f0, o[y].z *= f0, o[y].w *= f0;
            M[y] = m;
#pragma unroll
            for (int x = 0; x < kJoin; ++x) {
              if (c + x < n) {
                const float f = e[y][x].x == m ? 1.f : ex2_approx(e[y][x].x - m);
                L[y] += e[y][x].y * f;
                o[y].x += v[y][x].x * f, o[y].y += v[y][x].y * f;
                o[y].z += v[y][x].z * f, o[y].w += v[y][x].w * f;
              }
            }
          }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (y == 1 && i0 + kWarps * 32 >= items) continue;
          if (last) {
            const long long at = (long long)crow * a.R + q0 + qi[y];
            put4<F32>(a.out, at * D + dim, o[y], L[y]);
            if (a.lse && dim == 0) a.lse[at] = lse_of(M[y], L[y]);
          } else {  // in the first one's place; a thread writes the channels that it read, the sums follow
            *reinterpret_cast<float4*>(parts + (size_t)s0 * kPart + 2 * kAttnQ + qi[y] * D + dim) = o[y];
            if (dim == 0) ml[qi[y]] = make_float2(M[y], L[y]);
          }
        }
      }
      if (!last) {
        named_bar_sync(1, kWarps * 32);
        if ((int)threadIdx.x < nq) reinterpret_cast<float2*>(parts + (size_t)s0 * kPart)[threadIdx.x] = ml[threadIdx.x];
      }
    };
    // last_of for all threads; what they wrote before is seen by who is the last
    auto leave = [&](int* counter, int n) {
      named_bar_sync(1, kWarps * 32);
      if (threadIdx.x == 0) {
        __threadfence();  // what the barrier ordered before it is seen before the count
        *last_flag = last_of(counter, n, false);
        __threadfence();
      }
      named_bar_sync(1, kWarps * 32);
      return *last_flag;
    };
    const int whose = leave(arrived + first, in_eight);
    if (whose == kLost && eights > 1 && threadIdx.x == 0) last_of(arrived + 2 * gridDim.x + r, eights, true);
    if (whose != kJoined) continue;
    join(in_eight, first, 2 * (c_first + eight * kJoin + 1), 2, eights == 1);
    if (eights == 1 || leave(arrived + 2 * gridDim.x + r, eights) != kJoined) continue;
    join(eights, 2 * c_first + 1, 2 * (c_first + kJoin), 2 * kJoin, true);
  }
}

template <int D, int NG, int NT, bool F32>
int run(AttnArgs a, cudaStream_t st) {
  using S = Smem<D, NG, NT, F32>;
  auto k = paged_attn_kernel<D, NG, NT, F32>;
  static std::atomic<unsigned long long> ready{0};
  if (const int rc = allow_smem(k, S::kBytes, ready)) return rc;
  const int chunks = (a.R + S::NQ - 1) / S::NQ;
  const int per_sm = NT == 1 && !F32 ? kAttnCtasPerSm : 2;
  const int grid = max(1, sm_count() * per_sm / chunks);
  const int all = a.rows.n_rows;
  for (int r0 = 0; r0 < all; r0 += kAttnRows) {
    a.row0 = r0;
    a.n_rows = min(kAttnRows, all - r0);
    const int rc = launch_smem(k, dim3(grid, chunks), kThreads, S::kBytes, st, a);
    if (rc) return rc;
  }
  return KV_OK;
}

template <int D, int NG>
int run_as(const AttnArgs& a, bool f32, cudaStream_t st) {
  if (f32) return run<D, NG, 1, true>(a, st);
  return a.R <= 8 ? run<D, NG, 1, false>(a, st) : run<D, NG, 2, false>(a, st);
}

}  // namespace

int launch_paged_attn(const kv_paged_shape& sh, const PageGeom& g, const SeqRows& rows, const PagedCache& c,
                      uint8_t* ws, int n_q, const void* q, void* out, float* lse, cudaStream_t st) {
  AttnArgs a = {};
  a.g = g;
  a.rows = rows;
  a.c = c;
  a.n_q = n_q;
  a.group = sh.group;
  a.R = n_q * sh.group;
  a.scale2 = 1.4426950408889634f / sqrtf((float)sh.head_dim);
  a.inv_scale2 = 1.f / a.scale2;
  a.q = q;
  a.out = out;
  a.lse = lse;
  const PagedWs w = paged_ws_layout(sh);
  a.arrived = reinterpret_cast<int*>(ws + w.arrived);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.limit_ns = wait_limit_ns();
  a.kc = {0x43004300u, 0xc308c308u, 0x64006400u, 0x54005400u, 0xe408e408u, 0xd480d480u};
  const bool f32 = sh.dtype == KV_F32;
  if (g.d == 64) return g.G == 1 ? run_as<64, 1>(a, f32, st) : run_as<64, 2>(a, f32, st);
  return g.G == 1 ? run_as<128, 1>(a, f32, st) : g.G == 2 ? run_as<128, 2>(a, f32, st) : run_as<128, 4>(a, f32, st);
}

}  // namespace kvc

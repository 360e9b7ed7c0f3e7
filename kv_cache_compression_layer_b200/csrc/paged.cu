// The paged 4-bit KV cache: storing tokens (quantisation), reading them back,
// and forking, copying, compacting and freeing pages. Declarations and the
// formats are in include/kvcomp_paged.h; attention is in paged_attn.cu.
//
// A call that needs pages runs a plan kernel (one CTA) and a data kernel.
// The plan sums the rows' needs in call-row order, lists that many of the
// lowest free pages from the bitmap and refuses the rows that do not fit; the
// data kernel moves the tokens and, where it reaches the first token of a new
// page, enters the page into the row's list, its count and the bitmap. No
// device wait, no atomics whose order shows: a page's count is an integer sum
// and the bitmap a set. The plan is a chain of dependent loads and block sums
// of one CTA, 2.5 us for 288 rows; what bounds the others stands at each.
#include <climits>

#include "paged_common.cuh"

namespace kvc {

bool paged_shape_ok(const kv_paged_shape* sh) {
  if (!sh) return false;
  if (sh->n_seqs < 1 || sh->n_layers < 1 || sh->n_kv_heads < 1 || sh->group < 1 || sh->group > 16) return false;
  if (sh->n_seqs > KV_PAGED_MAX_ROWS || sh->n_layers > KV_PAGED_MAX_ROWS || sh->n_kv_heads > KV_PAGED_MAX_ROWS)
    return false;
  if ((long long)sh->n_layers * sh->n_kv_heads > KV_PAGED_MAX_ROWS) return false;
  if ((long long)sh->n_seqs * sh->n_layers * sh->n_kv_heads > KV_PAGED_MAX_ROWS) return false;
  if (sh->head_dim != 64 && sh->head_dim != 128) return false;
  if (sh->dtype != KV_BF16 && sh->dtype != KV_F32) return false;
  if (sh->quant_group != 32 && sh->quant_group != 64 && sh->quant_group != 128) return false;
  if (sh->quant_group > sh->head_dim) return false;
  if (sh->page_tokens != 16 && sh->page_tokens != 32 && sh->page_tokens != 64 && sh->page_tokens != 128) return false;
  if (sh->n_pages < 1 || sh->n_pages > KV_PAGED_MAX_PAGES) return false;
  if (sh->max_pages < 1 || (long long)sh->max_pages * sh->page_tokens > KV_PAGED_MAX_TOKENS) return false;
  return true;
}

PageGeom page_geom(const kv_paged_shape& sh) {
  PageGeom g;
  g.P = sh.page_tokens;
  g.log_p = sh.page_tokens == 16 ? 4 : sh.page_tokens == 32 ? 5 : sh.page_tokens == 64 ? 6 : 7;
  g.d = sh.head_dim;
  g.qg = sh.quant_group;
  g.G = sh.head_dim / sh.quant_group;
  g.v = g.P * g.d / 2;
  g.ks = 2 * g.v;
  g.vs = g.ks + g.P * g.G * 4;
  g.bytes = g.vs + g.P * g.G * 4;
  g.n_pages = sh.n_pages;
  g.max_pages = sh.max_pages;
  return g;
}

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

PagedWs paged_ws_layout(const kv_paged_shape& sh) {
  const size_t rows = (size_t)(sh.n_seqs < KV_MAX_SEQ ? sh.n_seqs : KV_MAX_SEQ) * sh.n_layers * sh.n_kv_heads;
  PagedWs w;
  w.arrived = 0;
  w.arrived_bytes =
      ((size_t)sm_count() * kAttnCtasPerSm * 2 + (KV_PAGED_MAX_QUERIES / 8) * kAttnRows) * sizeof(int);
  w.part = align256(w.arrived + w.arrived_bytes);
  // two partials per attention CTA: (max, sum) and the output of up to kAttnQ query rows
  w.plan = align256(w.part + (size_t)sm_count() * kAttnCtasPerSm * 2 * kAttnQ * (sh.head_dim + 2) * sizeof(float));
  w.unit = align256(w.plan + rows * sizeof(RowPlan));
  w.take = align256(w.unit + (rows + 1) * sizeof(int));
  w.bytes = align256(w.take + (size_t)sh.n_pages * sizeof(int));
  return w;
}

namespace {

constexpr int kPlanThreads = 1024;

enum PlanOp { kAppend, kFork, kCopy, kCompact };

struct PlanArgs {
  PageGeom g;         // of the cache that takes pages
  SeqRows dst, src;   // src: fork, copy, compact
  PagedCache c;       // the cache that takes pages
  const int32_t* src_len;
  int src_max;        // tokens a source row can hold at most
  const int32_t* count;
  int n_each;
  RowPlan* plan;
  int* unit;  // [rows + 1] units of kUnit tokens before each row (append, compact)
  int* take;
};

// Exclusive sum over the block in thread order; *total = the block's sum.
__device__ long long block_excl(long long v, long long* total, long long* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long t = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    sh[32 + lane] = t;
  }
  __syncthreads();
  *total = sh[63];
  return x - v + (warp ? sh[32 + warp - 1] : 0);
}

__device__ __forceinline__ int pages_of(const PageGeom& g, int tokens) { return (tokens + g.P - 1) >> g.log_p; }

template <int OP>
__global__ void __launch_bounds__(kPlanThreads, 1) paged_plan_kernel(const PlanArgs a) {
  __shared__ long long sh[64];
  const PageGeom& g = a.g;
  const int row_max = g.max_pages << g.log_p;  // tokens a row can hold
  pdl_launch_dependents();
  pdl_wait();
  int bad = 0;
  // needs of the rows, in order
  long long demand = 0;
  for (int i0 = 0; i0 < a.dst.n_rows; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    RowPlan p{0, -1, 0, 0};
    int need = 0;
    if (i < a.dst.n_rows) {
      const int tr = table_row(a.dst, i);
      const int held = a.c.len[tr];
      bool ok = held >= 0 && held <= row_max;
      if (!ok) bad |= KV_DEV_BOUNDS;
      if (OP == kAppend) {
        const int n = a.count ? max(0, a.count[i]) : a.n_each;
        p.old = held;
        p.n = n;
        if (ok && n > row_max - held) {
          ok = false;
          bad |= KV_DEV_CAPACITY;
        }
        if (ok) {
          p.fresh = pages_of(g, held);
          need = pages_of(g, held + n) - p.fresh;
        }
      } else {
        const int ts = table_row(a.src, i);
        const int sl = a.src_len[ts];
        if (sl < 0 || sl > a.src_max) {
          ok = false;
          bad |= KV_DEV_BOUNDS;
        }
        const bool in_place = OP == kCompact && ts == tr;
        if (ok && held != 0 && !in_place) {
          ok = false;
          bad |= KV_DEV_BUSY;
        }
        p.old = sl;
        p.n = OP == kCompact ? max(0, a.count[i]) : sl;
        if (ok && p.n > row_max) {
          ok = false;
          bad |= KV_DEV_CAPACITY;
        }
        if (ok) {
          p.fresh = OP == kFork ? p.n >> g.log_p : 0;
          need = pages_of(g, p.n) - p.fresh;
        }
      }
    }
    long long tot;
    const long long at = demand + block_excl(need, &tot, sh);
    if (i < a.dst.n_rows) {
      p.take = need == 0 ? 0 : (int)(at < INT_MAX ? at : INT_MAX);
      a.plan[i] = p;
    }
    demand += tot;
  }
  // the lowest `demand` free pages (or all of them), a word of the bitmap per thread
  long long found = 0;
  const int words = (g.n_pages + 31) >> 5;
  const int lane = threadIdx.x & 31;
  for (int w0 = 0; w0 < words && found < demand; w0 += kPlanThreads) {
    const int w = w0 + threadIdx.x;
    const uint32_t bits = w < words ? a.c.free_bits[w] : 0u;
    long long tot;
    const long long at = found + block_excl(__popc(bits), &tot, sh);
    for (int l = 0; l < 32; ++l) {  // the warp writes one lane's pages at a time
      const uint32_t b = __shfl_sync(0xffffffffu, bits, l);
      const long long r = __shfl_sync(0xffffffffu, at, l);
      if (r >= demand) break;
      const int rank = (int)r + __popc(b & ((1u << lane) - 1u));
      const int page = ((w - lane + l) << 5) + lane;
      if ((b >> lane) & 1u) {
        if (rank < demand && page < g.n_pages) a.take[rank] = page;
      }
    }
    found += tot;
  }
  // units of the rows that are served; lengths as they will be
  long long units = 0;
  for (int i0 = 0; i0 < a.dst.n_rows; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int u = 0;
    if (i < a.dst.n_rows) {
      RowPlan p = a.plan[i];
      if (p.fresh >= 0) {
        const int end = OP == kAppend ? p.old + p.n : p.n;
        const int need = pages_of(g, end) - p.fresh;
        if (need > 0 && (long long)p.take + need > found) {
          bad |= KV_DEV_PAGES;
          a.plan[i].fresh = -1;
        } else {
          a.c.len[table_row(a.dst, i)] = end;
          if (p.n > 0) u = OP == kAppend ? ((end + kUnit - 1) / kUnit - p.old / kUnit) : (end + kUnit - 1) / kUnit;
        }
      }
    }
    if (OP == kAppend || OP == kCompact) {
      long long tot;
      const long long at = units + block_excl(u, &tot, sh);
      if (i < a.dst.n_rows) a.unit[i] = (int)at;
      units += tot;
    }
  }
  if ((OP == kAppend || OP == kCompact) && threadIdx.x == 0) a.unit[a.dst.n_rows] = (int)units;
  if (bad) atomicOr(a.c.status, bad);
}

// Enters new page `page` as entry j of a row's list.
__device__ __forceinline__ void claim_page(const PagedCache& c, const PageGeom& g, int trow, int j, int page) {
  c.table[(size_t)trow * g.max_pages + j] = page;
  c.ref[page] = 1;
  atomicAnd(&c.free_bits[page >> 5], ~(1u << (page & 31)));
}

// Gives up one holder of a page.
__device__ __forceinline__ void drop_page(const PagedCache& c, const PageGeom& g, int page) {
  if (page < 0 || page >= g.n_pages) {
    atomicOr(c.status, KV_DEV_BOUNDS);
    return;
  }
  const int before = atomicSub(&c.ref[page], 1);
  if (before == 1) atomicOr(&c.free_bits[page >> 5], 1u << (page & 31));
  if (before < 1) {  // it had no holder: leave it free
    atomicAdd(&c.ref[page], 1);
    atomicOr(c.status, KV_DEV_BOUNDS);
  }
}

// The row that unit u lies in (unit[row] <= u < unit[row + 1]), by the whole
// warp: 32 probes a round. u < unit[n].
__device__ __forceinline__ int find_unit_row(const int* unit, int n, int u) {
  int lo = 0, hi = n;  // unit[lo] <= u, u < unit[hi]
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < hi && unit[at] <= u;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int last = 31 - __clz(m);  // lane 0 always holds
    const int nlo = lo + last * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

// ---------------------------------------------------------------- storing
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float bf16_round(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }
__device__ __forceinline__ uint32_t bf16_bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// What a lane holds of a quantised group: the codes of its 32 channels,
// channel 8 i + n in bits 4 n of w[i], and the packed (s, m).
struct Quantised {
  uint32_t w[4], scale;
};

// The same by the definition, in float64: the quotient's rounding does not
// reach a half (x, m and s have at most 24, 8 and 8 bits). Calls, so that the
// common path keeps its registers and its place in the instruction cache.
__device__ __noinline__ float step_exact(float mx, float m) {  // NaN: the group holds NaN
  if (!(fabsf(mx) < INFINITY && fabsf(m) < INFINITY)) return __uint_as_float(0x7fffffffu);
  return mx > m ? bf16_round((float)(((double)mx - (double)m) / 15.0)) : 0.f;
}
__device__ __noinline__ uint32_t codes_exact(float4 a, float4 b, float m, float s) {
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t w = 0;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const double q = ((double)x[n] - (double)m) / (double)s;
    w |= (uint32_t)rint(fmin(fmax(q, 0.0), 15.0)) << (4 * n);
  }
  return w;
}

// Two float32 in one register pair, and the packed operations on them.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Where 16-byte piece q of a part lies in shared memory: a lane's N pieces
// follow each other, and eight lanes' fall on different banks.
template <int N>
__device__ __forceinline__ int piece_at(int q) {
  return q ^ ((q >> 3) & (N - 1));
}

// Channels 8 i .. 8 i + 7 of the 32 that start at piece q of a part in shared memory.
template <bool F32>
__device__ __forceinline__ void eight(const uint4* part, int q, int i, float4& a, float4& b) {
  if constexpr (F32) {
    a = *reinterpret_cast<const float4*>(part + piece_at<8>(q + 2 * i));
    b = *reinterpret_cast<const float4*>(part + piece_at<8>(q + 2 * i + 1));
  } else {
    uint4 u;  // in order: taken early, they cost more registers than there are
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(smem_u32(part + piece_at<4>(q + i)))
                 : "memory");
    a = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                    __uint_as_float(u.y & 0xffff0000u));
    b = make_float4(__uint_as_float(u.z << 16), __uint_as_float(u.z & 0xffff0000u), __uint_as_float(u.w << 16),
                    __uint_as_float(u.w & 0xffff0000u));
  }
}

// Quantises the 32 channels that a lane holds of a group with largest value mx
// and base m (bf16 of the smallest), to exact arithmetic's result; false where
// it may not be. The step: the float32 product is off by a few of its last
// bits, which matters next to the middle of two bf16. The codes: x - m is exact
// in float32 unless the two lie far apart, and q follows from a reciprocal by
// one correction with the exact remainder. An exact quotient k + 1/2 comes out
// as that; another differs from it by the last bit of x - m over s at least,
// which is more than half the last bit of q by 1 part in 255 (s has 8 bits), so
// it comes out on its own side. What this does not cover: a step next to a
// middle, tiny, zero or not finite; an x - m that was rounded. For F32 that is
// common, and matters only with a quotient within 1e-5 of a half. bf16 numbers
// are multiples of 2^-8 of themselves, so none is rounded while the smallest
// magnitude but 0 (`least`: of these 32) is 2^-16 of mx - m or more; where it is
// not, each channel is looked at.
template <bool F32>
__device__ __forceinline__ bool quantise_fast(const uint4* part, int q0, float mx, float m, float least, Quantised& res) {
  const float magic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, in the low bits of the sum
  const float f = __fmul_rn(__fsub_rn(mx, m), 1.f / 15.f);
  const float s = bf16_round(f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  const uint64_t m2 = f2(m, m), nm2 = f2(-m, -m), r2 = f2(r, r), ns2 = f2(-s, -s), g2 = f2(magic, magic),
                 n1 = f2(-1.f, -1.f);
  uint32_t off = 0;
  float dev = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 a, b;
    eight<F32>(part, q0, i, a, b);
    const uint64_t x[4] = {f2(a.x, a.y), f2(a.z, a.w), f2(b.x, b.y), f2(b.z, b.w)};
    uint32_t w = 0;
#pragma unroll
    for (int n = 3; n >= 0; --n) {
      const uint64_t v = x[n];
      const uint64_t t = add2(v, nm2);
      const uint64_t p = mul2(t, r2);
      uint64_t q = fma2(fma2(p, ns2, t), r2, p);
      if (F32) {  // the base may be above the smallest
        float c, d;
        unpack2(q, c, d);
        q = f2(fmaxf(c, 0.f), fmaxf(d, 0.f));
      }
      const uint64_t y = add2(q, g2);
      float y0, y1;
      unpack2(y, y0, y1);
      if (F32) {
        float c, d, e0, e1;
        unpack2(fma2(add2(y, f2(-magic, -magic)), n1, q), c, d);
        dev = fmaxf(dev, fmaxf(fabsf(c), fabsf(d)));
        // both 0 where t is exact; the first is not 0 where it was rounded and |x| <= |m|, the second where |x| >= |m|
        unpack2(fma2(v, n1, add2(t, m2)), e0, e1);
        off |= __float_as_uint(e0) | __float_as_uint(e1);
        unpack2(add2(fma2(v, n1, t), m2), e0, e1);
        off |= __float_as_uint(e0) | __float_as_uint(e1);
      }
      w = (w << 4) + __float_as_uint(y1);
      w = (w << 4) + __float_as_uint(y0);
    }
    res.w[i] = w - 0x3F400000u;  // what the eight shifted exponents of `magic` (0x4B400000) add up to
  }
  res.scale = bf16_bits(f) | (__float_as_uint(m) & 0xffff0000u);
  if (!F32 && (least < __fsub_rn(mx, m) * 0x1p-16f || (m != 0.f && fabsf(m) < __fsub_rn(mx, m) * 0x1p-16f))) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      float4 a, b;
      eight<F32>(part, q0, i, a, b);
      const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int n = 0; n < 8; ++n) {  // t is exact where both are 0
        const float t = __fsub_rn(x[n], m);
        off |= __float_as_uint(__fsub_rn(__fadd_rn(t, m), x[n])) | __float_as_uint(__fadd_rn(__fsub_rn(t, x[n]), m));
      }
    }
  }
  return f > 1e-30f && f < 1e37f && (__float_as_uint(f) & 0xffffu) - 0x7fe0u > 0x40u &&
         ((off & 0x7fffffffu) == 0u || (F32 && dev <= 0.49999f));
}

template <bool F32>
__device__ __forceinline__ void quantise_exact(const uint4* part, int q, float mx, float m, Quantised& res) {
  const float s = step_exact(mx, m);
  res.scale = s == s ? bf16_bits(s) | (__float_as_uint(m) & 0xffff0000u) : 0x7fff7fffu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 a, b;
    eight<F32>(part, q, i, a, b);
    res.w[i] = s > 0.f ? codes_exact(a, b, m, s) : 0u;
  }
}

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The number of smaller magnitude of each pair (its sign is the product's).
__device__ __forceinline__ uint32_t min2_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Of N rows (the 32 channels from piece q + n * dq on each): the largest value
// of the group that the LG consecutive lanes hold, and bf16 of its smallest
// (NaN and infinities reach them); bf16: the least magnitude of the 32 channels.
template <bool F32, int LG, int N>
__device__ __forceinline__ void group_ends(const uint4* part, int q, int dq, float (&mx)[N], float (&m)[N],
                                           float (&least)[N]) {
  if constexpr (F32) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4 a, b;
        eight<true>(part, q + n * dq, i, a, b);
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (i == 0) mx[n] = m[n] = x[0];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          mx[n] = max_nan(mx[n], x[k]);
          m[n] = min_nan(m[n], x[k]);
        }
      }
    }
#pragma unroll
    for (int o = 1; o < LG; o <<= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        mx[n] = max_nan(mx[n], __shfl_xor_sync(0xffffffffu, mx[n], o));
        m[n] = min_nan(m[n], __shfl_xor_sync(0xffffffffu, m[n], o));
      }
#pragma unroll
    for (int n = 0; n < N; ++n) m[n] = bf16_round(m[n]);
  } else {
    uint32_t v[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t hi = 0, lo = 0, near = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 u = part[piece_at<4>(q + n * dq + i)];
        const uint32_t h = max2_nan(max2_nan(u.x, u.y), max2_nan(u.z, u.w));
        const uint32_t l = min2_nan(min2_nan(u.x, u.y), min2_nan(u.z, u.w));
        hi = i ? max2_nan(hi, h) : h;
        lo = i ? min2_nan(lo, l) : l;
        const uint32_t k = min2_abs(min2_abs(u.x, u.y), min2_abs(u.z, u.w));
        near = i ? min2_abs(near, k) : k;
      }
      least[n] = fminf(fabsf(__uint_as_float(near << 16)), fabsf(__uint_as_float(near & 0xffff0000u)));
      lo ^= 0x80008000u;  // the largest and the negated smallest share a register
      v[n] = max2_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
    }
#pragma unroll
    for (int o = 1; o < LG; o <<= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = max2_nan(v[n], __shfl_xor_sync(0xffffffffu, v[n], o));
#pragma unroll
    for (int n = 0; n < N; ++n) {
      mx[n] = __uint_as_float(v[n] << 16);
      m[n] = __uint_as_float((v[n] & 0xffff0000u) ^ 0x80000000u);
    }
  }
}

// Writes the 8 channels of codes w as m + c s, rounded once, with 16-byte
// stores. bf16: bits 0-3 of a half or-ed into 0x4300 are 128 + c, so two
// channels take a subtraction and a multiply-add in bf16. float32: the code
// or-ed into 2^23. `bits` is 0x43004300 or 0x4B000000.
template <bool F32>
__device__ __forceinline__ void store8(void* base, long long row, int d, int l, uint32_t w, uint32_t scale,
                                       uint32_t bits) {
  if constexpr (F32) {
    const float s = __uint_as_float(scale << 16), m = __uint_as_float(scale & 0xffff0000u);
    float x[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = fmaf(__uint_as_float(pick<15u>(w >> (4 * n), bits)) - 8388608.f, s, m);
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + row * d) + 2 * l;
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    const uint32_t s2 = __byte_perm(scale, 0, 0x1010), m2 = __byte_perm(scale, 0, 0x3232);
    uint32_t v[4];  // channels n and n + 4
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const uint32_t c = pick<0x000f000fu>(w >> (4 * n), bits);
      uint32_t e;
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(e) : "r"(c), "r"(bits));
      asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[n]) : "r"(e), "r"(s2), "r"(m2));
    }
    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + row * d)[l] =
        make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                   __byte_perm(v[2], v[3], 0x7632));
  }
}

constexpr int kMoveWarps = 8;

struct StoreArgs {
  PageGeom g;
  SeqRows rows;
  PagedCache c;
  const void* K;
  const void* V;
  long long n_src;
  int n_each;
  const int64_t* src_off;
  const int32_t* idx;
  const int64_t* idx_off;
  const RowPlan* plan;
  const int* unit;
  const int* take;
};

// Warps take runs of units of 16 tokens (a unit starts at a multiple of 16 of
// the row's tokens, so it lies in one page). D / 32 lanes hold a token's row, 32
// channels each (so that a group's scale, worked out in each of its lanes, is
// shared by 32 channels). The next part's (K's or V's) 16-byte pieces are on
// their way into shared memory while a part is quantised, and the next unit's
// place and source positions are read a part before those are needed. A part is
// quantised into shared memory in the page's layout and written with 16-byte
// stores (each part of a unit is contiguous).
//
// What bounds it: instructions, and their latency where registers allow 16 warps
// an SM. 1.93 M tokens of bf16, d = 128, kept at random from rows four times as
// long: 283 us for 1.27 GB (4.5 TB/s). A copy that did not quantise took 215.
// With 16 channels a lane loaded into registers, rows one after the other, three
// CTAs an SM: 325 us; with these side by side at 80 registers (they spill) 385,
// at 128 and two CTAs 340.
template <int D, int QG, bool F32>
struct StoreSmem {
  static constexpr int kPieces = F32 ? 8 : 4;                     // of a lane's 32 channels
  static constexpr int kSrc = kUnit * D * (F32 ? 4 : 2);          // a part's source rows, piece by piece
  static constexpr int kCode = kUnit * D / 2, kScale = kUnit * (D / QG) * 4;
  static constexpr int kWarp = 2 * kSrc + kCode + kScale, kBytes = kMoveWarps * kWarp;
};

// By what the RC 16-byte pieces of token t's codes change places in the stage.
template <int RC>
__device__ __forceinline__ int turn(int t) {
  return RC == 4 ? (t >> 1) & 3 : (t >> 2) & 1;
}

template <int D, int QG, bool F32>
__global__ void __launch_bounds__(kMoveWarps * 32, F32 ? 1 : 2) paged_store_kernel(const StoreArgs a) {
  using S = StoreSmem<D, QG, F32>;
  constexpr int G = D / QG, W = D / 32, TPI = 32 / W, ITER = kUnit / TPI, LG = QG / 32;
  constexpr int kCode = S::kCode, PC = S::kPieces;
  constexpr int RC = D / 2 / 16;  // 16-byte pieces of a token's codes
  extern __shared__ __align__(128) uint8_t smem[];
  const PageGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % W, sub = lane / W;
  pdl_launch_dependents();
  pdl_wait();
  const int n_rows = a.rows.n_rows;
  const int total = a.unit[n_rows];
  const long long nw = (long long)gridDim.x * kMoveWarps, w = (long long)blockIdx.x * kMoveWarps + warp;
  const int u0 = (int)(w * total / nw), u1 = (int)((w + 1) * total / nw);
  if (u0 >= u1) return;
  uint4* in = reinterpret_cast<uint4*>(smem + warp * S::kWarp);
  uint8_t* st = smem + warp * S::kWarp + 2 * S::kSrc;
  int bad = 0;
  // the row of the next unit: its units [row_u0, row_u1), plan and source
  int row = -1, row_u0 = 0, row_u1 = -1;
  RowPlan p{};
  long long base = 0, at = 0;

  // A unit: where it goes (page, place of its first token, its new tokens [f, e)).
  struct Unit {
    int page, place, f, e;
  };
  Unit now, next{};
  int spot = 0;        // in lane t, the source position of the next unit's token t
  bool isnew = false;  // the next unit's page is new
  auto locate = [&](int u) {
    if (u >= row_u1) {
      row = find_unit_row(a.unit, n_rows, u);
      row_u0 = a.unit[row];
      row_u1 = a.unit[row + 1];
      p = a.plan[row];
      base = a.src_off ? a.src_off[row] : (long long)row * a.n_each;
      if (a.idx) at = a.idx_off[row];
    }
    const int pos0 = (p.old / kUnit + u - row_u0) * kUnit;
    next.f = max(p.old - pos0, 0);
    next.e = min(kUnit, p.old + p.n - pos0);
    const int j = pos0 >> g.log_p;
    next.place = pos0 & (g.P - 1);
    isnew = j >= p.fresh;
    next.page = isnew ? a.take[p.take + j - p.fresh] : a.c.table[(size_t)table_row(a.rows, row) * g.max_pages + j];
    spot = pos0 + lane - p.old;
    if (a.idx && lane >= next.f && lane < next.e) spot = a.idx[at + spot];
  };
  // The byte offset of the source row of the next unit's token t in lane t (-1: none); enters a new page.
  auto settle = [&](int u) {
    if (isnew) {
      if (next.place == 0 && lane == 0)
        claim_page(a.c, g, table_row(a.rows, row), ((p.old / kUnit + u - row_u0) * kUnit) >> g.log_p, next.page);
    } else if (next.page < 0 || next.page >= g.n_pages) {
      bad |= KV_DEV_BOUNDS;
      next.f = next.e = 0;  // nothing of it is stored
      next.page = 0;
    }
    if (lane < next.f || lane >= next.e) return -1ll;
    const long long src = base + spot;
    if (src >= 0 && src < a.n_src) return src * (D * (F32 ? 4 : 2));
    bad |= KV_DEV_RANGE;
    return -1ll;
  };
  constexpr int PPR = W * PC;  // pieces of a row, at most 32
  const int mine = lane % PPR * 16;
  auto fetch = [&](uint4* part, const void* from, long long src) {
    const uint8_t* base = static_cast<const uint8_t*>(from) + mine;
#pragma unroll
    for (int x = 0; x < kUnit * PPR / 32; ++x) {
      const long long s = __shfl_sync(0xffffffffu, src, x * (32 / PPR) + lane / PPR);
      // a piece that has no source is zeros: none of its bytes are read
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(part + piece_at<PC>(x * 32 + lane))),
                   "l"(s >= 0 ? base + s : reinterpret_cast<const uint8_t*>(a.unit)), "r"(s >= 0 ? 16 : 0)
                   : "memory");
    }
  };

  locate(u0);
  long long src = settle(u0);
  now = next;
  fetch(in, a.K, src);
#pragma unroll 1
  for (int i = 2 * u0; i < 2 * u1; ++i) {
    const bool v = i & 1;  // the unit's V, else its K
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();  // the part is there, the previous one is done with
    const uint4* part = in + (v ? S::kSrc / 16 : 0);
    const Unit here = now;
    if (!v) {
      fetch(in + S::kSrc / 16, a.V, src);
      if (i + 2 < 2 * u1) locate((i >> 1) + 1);
    } else if (i + 1 < 2 * u1) {
      src = settle((i >> 1) + 1);
      now = next;
      fetch(in, a.K, src);
    }
    // the rows side by side, what the fast way does not cover afterwards: a branch for each would keep them apart
    float mx[ITER], m[ITER], least[ITER];
    Quantised z[ITER];
    unsigned hard = 0;
    group_ends<F32, LG>(part, lane * PC, 32 * PC, mx, m, least);
#pragma unroll
    for (int it = 0; it < ITER; ++it)
      if (!quantise_fast<F32>(part, (it * 32 + lane) * PC, mx[it], m[it], least[it], z[it])) hard |= 1u << it;
    if (hard) {
#pragma unroll
      for (int it = 0; it < ITER; ++it)
        if (hard >> it & 1) quantise_exact<F32>(part, (it * 32 + lane) * PC, mx[it], m[it], z[it]);
    }
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      // channels 32 l + 8 i + n are word (i, l) of K, or the 16-bit words (2 i, l) and (2 i + 1, l) of V, in places
      // swapped by the token's bit 1; 16-byte pieces of the stage are turned by the token so that banks differ
      const int t = it * TPI + sub;
      uint8_t* row_st = st + t * (D / 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at_byte = v ? ((2 * i) ^ ((t & 2) << 1)) * (2 * W) + 2 * l : i * (4 * W) + 4 * l;
        uint8_t* to = row_st + (((at_byte >> 4) ^ turn<RC>(t)) << 4) + (at_byte & 15);
        if (!v) {
          *reinterpret_cast<uint32_t*>(to) = z[it].w[i];
        } else {
          reinterpret_cast<uint16_t*>(to)[0] = (uint16_t)z[it].w[i];
          reinterpret_cast<uint16_t*>(to)[W] = (uint16_t)(z[it].w[i] >> 16);
        }
      }
      if (l % LG == 0) reinterpret_cast<uint32_t*>(st + kCode)[t * G + l / LG] = z[it].scale;
    }
    __syncwarp();
    uint8_t* pg = a.c.pages + (size_t)here.page * g.bytes;
    const uint4* ss = reinterpret_cast<const uint4*>(st);
    uint4* d = reinterpret_cast<uint4*>(pg + (v ? g.v : 0) + here.place * (D / 2));
    const uint32_t* sx = reinterpret_cast<const uint32_t*>(st + kCode);
    uint32_t* dx = reinterpret_cast<uint32_t*>(pg + (v ? g.vs : g.ks)) + here.place * G;
#pragma unroll
    for (int x = lane; x < kUnit * RC; x += 32)
      if (x >= here.f * RC && x < here.e * RC) d[x] = ss[x ^ turn<RC>(x / RC)];
#pragma unroll
    for (int x = lane; x < (kUnit * G + 31) / 32 * 32; x += 32)
      if (x >= here.f * G && x < here.e * G) dx[x] = sx[x];
  }
  if (bad) atomicOr(a.c.status, bad);
}

// ---------------------------------------------------------------- reading
struct LoadArgs {
  PageGeom g;
  SeqRows rows;
  PagedCache c;
  const int64_t* out_off;
  long long n_out;
  void* K;
  void* V;
  uint32_t bits;  // see store8
};

// Warps take runs of 16 output rows; lane t finds the token of output row t.
// What bounds it: the writes, 512 of 656 bytes a token at d = 128 in bf16. 1.93 M
// tokens take 270 us; a fill of the 990 MB written takes 256 us (3.87 TB/s).
template <int D, int QG, bool F32>
__global__ void __launch_bounds__(kMoveWarps * 32, 4) paged_load_kernel(const LoadArgs a) {
  constexpr int G = D / QG, LT = D / 8, TPI = 32 / LT, ITER = kUnit / TPI, W = D / 32;
  const PageGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LT, sub = lane / LT;
  pdl_launch_dependents();
  pdl_wait();
  const int n_rows = a.rows.n_rows;
  int bad = 0;
  const long long first = a.out_off[0], last_ = a.out_off[n_rows];
  const long long lo = max(first, 0ll), hi = min(last_, a.n_out);
  if (first < 0 || last_ > a.n_out) bad |= KV_DEV_RANGE;
  const long long units = hi > lo ? (hi - lo + kUnit - 1) / kUnit : 0;
  const long long nw = (long long)gridDim.x * kMoveWarps, w = (long long)blockIdx.x * kMoveWarps + warp;
  const long long u0 = w * units / nw, u1 = (w + 1) * units / nw;
  int row = 0;
  long long r0 = 0, r1 = -1;  // out_off of the row and of the next
  for (long long u = u0; u < u1; ++u) {
    const long long o0 = lo + u * kUnit, o = o0 + lane;
    const uint8_t* pg = nullptr;
    int place = 0;
    if (lane < kUnit && o < hi) {
      if (!(o >= r0 && o < r1)) {  // the last row that starts at or before o
        int x = 0, y = n_rows - 1;
        while (x < y) {
          const int mid = (x + y + 1) >> 1;
          if (a.out_off[mid] <= o) x = mid;
          else y = mid - 1;
        }
        row = x;
        r0 = a.out_off[row];
        r1 = a.out_off[row + 1];
      }
      const int trow = table_row(a.rows, row);
      const long long t = o - r0;
      const int held = a.c.len[trow];
      if (held < 0 || held > (g.max_pages << g.log_p)) bad |= KV_DEV_BOUNDS;
      else if (t >= 0 && t < held && o < r1) {
        const int page = a.c.table[(size_t)trow * g.max_pages + (t >> g.log_p)];
        place = (int)(t & (g.P - 1));
        if (page < 0 || page >= g.n_pages) bad |= KV_DEV_BOUNDS;
        else pg = a.c.pages + (size_t)page * g.bytes;
      }
    }
    uint32_t kc[ITER], vc[ITER], ksc[ITER], vsc[ITER];
    bool have[ITER];
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int t = it * TPI + sub;
      const uint8_t* q = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(pg), t));
      const int pl = __shfl_sync(0xffffffffu, place, t);
      have[it] = q != nullptr;
      kc[it] = vc[it] = ksc[it] = vsc[it] = 0;
      if (have[it]) {
        kc[it] = reinterpret_cast<const uint32_t*>(q + pl * (D / 2))[(l & 3) * W + (l >> 2)];
        const int pv = (2 * (l & 3)) ^ ((pl & 2) << 1);
        const uint16_t* hv = reinterpret_cast<const uint16_t*>(q + g.v + pl * (D / 2)) + pv * W + (l >> 2);
        vc[it] = (uint32_t)hv[0] | ((uint32_t)hv[W] << 16);
        ksc[it] = reinterpret_cast<const uint32_t*>(q + g.ks)[pl * G + l / (QG / 8)];
        vsc[it] = reinterpret_cast<const uint32_t*>(q + g.vs)[pl * G + l / (QG / 8)];
      }
    }
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      if (!have[it]) continue;
      const long long orow = o0 + it * TPI + sub;
      store8<F32>(a.K, orow, D, l, kc[it], ksc[it], a.bits);
      store8<F32>(a.V, orow, D, l, vc[it], vsc[it], a.bits);
    }
  }
  if (bad) atomicOr(a.c.status, bad);
}

// ---------------------------------------------------------- moving pages
struct MoveArgs {
  PageGeom g;     // of the destination
  SeqRows dst, src;
  PagedCache c;   // destination
  const uint8_t* src_pages;
  const int32_t* src_table;
  int src_n_pages, src_max_pages;
  const int32_t* idx;
  const int64_t* idx_off;
  const RowPlan* plan;
  const int* unit;
  const int* take;
};

constexpr int kRowThreads = 256;

// Copies a page (a multiple of 16 bytes) with the whole block.
__device__ __forceinline__ void copy_page(uint8_t* dst, const uint8_t* src, int bytes) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  const int n = bytes / 16;
  for (int i = threadIdx.x; i < n; i += 4 * kRowThreads) {
    uint4 v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i + x * kRowThreads < n) v[x] = s[i + x * kRowThreads];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i + x * kRowThreads < n) d[i + x * kRowThreads] = v[x];
  }
}

// One CTA per destination row: the full pages gain a holder, the rest is copied. Latency: a fork of
// 288 rows of 1500 tokens and its freeing take 11 us.
__global__ void __launch_bounds__(kRowThreads) paged_fork_kernel(const MoveArgs a) {
  const PageGeom& g = a.g;
  const int row = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const RowPlan p = a.plan[row];
  if (p.fresh < 0) return;
  const int td = table_row(a.dst, row), ts = table_row(a.src, row);
  const int32_t* from = a.src_table + (size_t)ts * a.src_max_pages;
  int32_t* to = a.c.table + (size_t)td * g.max_pages;
  for (int j = threadIdx.x; j < p.fresh; j += kRowThreads) {
    const int page = from[j];
    to[j] = page;
    if (page < 0 || page >= g.n_pages) atomicOr(a.c.status, KV_DEV_BOUNDS);
    else atomicAdd(&a.c.ref[page], 1);
  }
  if (p.n & (g.P - 1)) {
    const int page = from[p.fresh], fresh = a.take[p.take];
    if (threadIdx.x == 0) claim_page(a.c, g, td, p.fresh, fresh);
    if (page < 0 || page >= g.n_pages) {
      if (threadIdx.x == 0) atomicOr(a.c.status, KV_DEV_BOUNDS);
    } else {
      copy_page(a.c.pages + (size_t)fresh * g.bytes, a.src_pages + (size_t)page * g.bytes, g.bytes);
    }
  }
}

// Every page of a row into a new one: grid (rows, slices); a slice's CTA takes every gridDim.y-th page. Bound by
// HBM: 26 us for 137 MB moved (5.3 TB/s).
__global__ void __launch_bounds__(kRowThreads) paged_copy_kernel(const MoveArgs a) {
  const PageGeom& g = a.g;
  const int row = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const RowPlan p = a.plan[row];
  if (p.fresh < 0) return;
  const int td = table_row(a.dst, row), ts = table_row(a.src, row);
  const int np = pages_of(g, p.n);
  for (int j = blockIdx.y; j < np; j += gridDim.y) {
    const int page = a.src_table[(size_t)ts * a.src_max_pages + j], fresh = a.take[p.take + j];
    if (threadIdx.x == 0) claim_page(a.c, g, td, j, fresh);
    if (page < 0 || page >= a.src_n_pages) {
      if (threadIdx.x == 0) atomicOr(a.c.status, KV_DEV_BOUNDS);
    } else {
      copy_page(a.c.pages + (size_t)fresh * g.bytes, a.src_pages + (size_t)page * g.bytes, g.bytes);
    }
  }
}

// The kept tokens' codes and scales into the new pages, in units of 16 of the
// tokens to be; a V row whose place differs in bit 1 has its halves swapped.
// The lists change hands in paged_commit_kernel, when every token has moved. 64-byte rows picked at random: 48 us for
// half of 1.23 M tokens, DRAM delivering the source pages whole (168 MB for 88).
__global__ void __launch_bounds__(kMoveWarps * 32) paged_compact_kernel(const MoveArgs a) {
  const PageGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int n_rows = a.dst.n_rows;
  const int total = a.unit[n_rows];
  const long long nw = (long long)gridDim.x * kMoveWarps, w = (long long)blockIdx.x * kMoveWarps + warp;
  const int u0 = (int)(w * total / nw), u1 = (int)((w + 1) * total / nw);
  if (u0 >= u1) return;
  const int rb = g.d / 2, rc = rb / 16;  // bytes and 16-byte pieces of a token's codes
  int row = find_unit_row(a.unit, n_rows, u0);
  int bad = 0;
  for (int u = u0; u < u1; ++u) {
    if (u >= a.unit[row + 1]) row = find_unit_row(a.unit, n_rows, u);
    const RowPlan p = a.plan[row];
    const int ts = table_row(a.src, row);
    const int pos0 = (u - a.unit[row]) * kUnit, n = min(kUnit, p.n - pos0);
    const int fresh = a.take[p.take + (pos0 >> g.log_p)], place0 = pos0 & (g.P - 1);
    const uint8_t* from = nullptr;
    int place = 0;
    if (lane < n) {
      const int pos = a.idx[a.idx_off[row] + pos0 + lane];
      if (pos < 0 || pos >= p.old) {
        bad |= KV_DEV_RANGE;
      } else {
        const int page = a.src_table[(size_t)ts * a.src_max_pages + (pos >> g.log_p)];
        place = pos & (g.P - 1);
        if (page < 0 || page >= g.n_pages) bad |= KV_DEV_BOUNDS;
        else from = a.src_pages + (size_t)page * g.bytes;
      }
    }
    uint8_t* to = a.c.pages + (size_t)fresh * g.bytes;
    // 32 / rc tokens at a time (8 for d = 128, 16 for d = 64), a lane per piece
    const int tpi = 32 / rc;
    const int piece = lane & (rc - 1), sub = lane / rc;
    for (int t0 = 0; t0 < n; t0 += tpi) {
      const int t = t0 + sub;
      const uint8_t* f = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), t & 31));
      const int pl = __shfl_sync(0xffffffffu, place, t & 31);
      if (t < n) {
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        const int to_place = place0 + t;
        if (f) {
          k = reinterpret_cast<const uint4*>(f + pl * rb)[piece];
          const int vp = piece ^ (((pl ^ to_place) & 2) ? rc / 2 : 0);
          v = reinterpret_cast<const uint4*>(f + g.v + pl * rb)[vp];
        }
        reinterpret_cast<uint4*>(to + to_place * rb)[piece] = k;
        reinterpret_cast<uint4*>(to + g.v + to_place * rb)[piece] = v;
      }
    }
    for (int i0 = 0; i0 < n * g.G; i0 += 32) {
      const int i = i0 + lane, t = i / g.G, x = i - t * g.G;
      const uint8_t* f = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), t & 31));
      const int pl = __shfl_sync(0xffffffffu, place, t & 31);
      if (i < n * g.G) {
        const uint32_t ks = f ? reinterpret_cast<const uint32_t*>(f + g.ks)[pl * g.G + x] : 0u;
        const uint32_t vs = f ? reinterpret_cast<const uint32_t*>(f + g.vs)[pl * g.G + x] : 0u;
        reinterpret_cast<uint32_t*>(to + g.ks)[place0 * g.G + i] = ks;
        reinterpret_cast<uint32_t*>(to + g.vs)[place0 * g.G + i] = vs;
      }
    }
  }
  if (bad) atomicOr(a.c.status, bad);
}

// After a compaction: a row replaced in place gives up its former pages, and the new ones enter the lists.
__global__ void __launch_bounds__(kRowThreads) paged_commit_kernel(const MoveArgs a) {
  const PageGeom& g = a.g;
  const int row = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const RowPlan p = a.plan[row];
  if (p.fresh < 0) return;
  const int td = table_row(a.dst, row);
  const int had = td == table_row(a.src, row) ? pages_of(g, p.old) : 0, has = pages_of(g, p.n);
  for (int j = threadIdx.x; j < max(had, has); j += kRowThreads) {
    if (j < had) drop_page(a.c, g, a.c.table[(size_t)td * g.max_pages + j]);
    if (j < has) claim_page(a.c, g, td, j, a.take[p.take + j]);
  }
}

// One CTA per row.
__global__ void __launch_bounds__(kRowThreads)
    paged_free_kernel(const PageGeom g, const SeqRows rows, const PagedCache c) {
  const int trow = table_row(rows, blockIdx.x);
  pdl_launch_dependents();
  pdl_wait();
  const int held = c.len[trow];
  if (held < 0 || held > (g.max_pages << g.log_p)) {
    if (threadIdx.x == 0) atomicOr(c.status, KV_DEV_BOUNDS);
    return;
  }
  const int np = pages_of(g, held);
  for (int j = threadIdx.x; j < np; j += kRowThreads) drop_page(c, g, c.table[(size_t)trow * g.max_pages + j]);
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) c.len[trow] = 0;
}

__global__ void __launch_bounds__(kRowThreads)
    paged_count_kernel(const PageGeom g, int n_rows, const PagedCache c) {
  for (int row = blockIdx.x; row < n_rows; row += gridDim.x) {
    const int held = c.len[row];
    if (held < 0 || held > (g.max_pages << g.log_p)) {
      if (threadIdx.x == 0) atomicOr(c.status, KV_DEV_BOUNDS);
      continue;
    }
    const int np = pages_of(g, held);
    for (int j = threadIdx.x; j < np; j += kRowThreads) {
      const int page = c.table[(size_t)row * g.max_pages + j];
      if (page < 0 || page >= g.n_pages) atomicOr(c.status, KV_DEV_BOUNDS);
      else atomicAdd(&c.ref[page], 1);
    }
  }
}

__global__ void __launch_bounds__(kRowThreads) paged_bits_kernel(int n_pages, const PagedCache c) {
  const int words = (n_pages + 31) >> 5;
  const int lane = threadIdx.x & 31;
  const int nw = (gridDim.x * kRowThreads) >> 5;
  for (int w = (blockIdx.x * kRowThreads + threadIdx.x) >> 5; w < words; w += nw) {
    const int page = (w << 5) + lane;
    const unsigned b = __ballot_sync(0xffffffffu, page < n_pages && c.ref[page] == 0);
    if (lane == 0) c.free_bits[w] = b;
  }
}

// ------------------------------------------------------------------- host
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
template <class T>
bool list_ok(const T* p) {  // aligned to its type, or none
  return (reinterpret_cast<uintptr_t>(p) & (sizeof(T) - 1)) == 0;
}

bool cache_ok(const kv_paged_cache* c) {
  return c && aligned16(c->pages) && aligned16(c->table) && aligned16(c->len) && aligned16(c->ref) &&
         aligned16(c->free_bits) && c->status && (reinterpret_cast<uintptr_t>(c->status) & 3) == 0;
}

PagedCache cache_of(const kv_paged_cache& c) {
  return {static_cast<uint8_t*>(c.pages), c.table, c.len, c.ref, c.free_bits, c.status};
}

// The rows of a call; false when a sequence or layer is outside the cache, or (distinct) named twice.
bool make_rows(const kv_paged_shape& sh, const int32_t* seq, int32_t n, int layer0, int n_lay, bool distinct,
               SeqRows* r) {
  if (!seq || n < 1 || n > KV_MAX_SEQ) return false;
  if (layer0 < 0 || n_lay < 1 || layer0 > sh.n_layers - n_lay) return false;
  for (int i = 0; i < n; ++i) {
    if (seq[i] < 0 || seq[i] >= sh.n_seqs) return false;
    if (distinct)
      for (int j = 0; j < i; ++j)
        if (seq[j] == seq[i]) return false;
  }
  r->n_seq = n;
  r->per_seq = n_lay * sh.n_kv_heads;
  r->first = layer0 * sh.n_kv_heads;
  r->table_rps = sh.n_layers * sh.n_kv_heads;
  r->n_rows = n * r->per_seq;
  for (int i = 0; i < KV_MAX_SEQ; ++i) r->seq[i] = i < n ? seq[i] : 0;
  return true;
}

template <int D, int QG, bool F32>
int store_with(int blocks, const StoreArgs& a, cudaStream_t st) {
  using S = StoreSmem<D, QG, F32>;
  auto k = paged_store_kernel<D, QG, F32>;
  static std::atomic<unsigned long long> ready{0};
  if (const int rc = allow_smem(k, S::kBytes, ready)) return rc;
  const int cap = (F32 ? 1 : 2) * sm_count();  // all resident
  return launch_smem(k, blocks < cap ? blocks : cap, kMoveWarps * 32, S::kBytes, st, a);
}
template <int D, int QG>
int store_as(bool f32, int blocks, const StoreArgs& a, cudaStream_t st) {
  return f32 ? store_with<D, QG, true>(blocks, a, st) : store_with<D, QG, false>(blocks, a, st);
}
template <int D, int QG>
int load_as(bool f32, int grid, const LoadArgs& a, cudaStream_t st) {
  return f32 ? launch(paged_load_kernel<D, QG, true>, grid, kMoveWarps * 32, st, a)
             : launch(paged_load_kernel<D, QG, false>, grid, kMoveWarps * 32, st, a);
}

struct Ws {
  RowPlan* plan;
  int* unit;
  int* take;
};
Ws ws_of(const kv_paged_shape& sh, void* ws) {
  const PagedWs w = paged_ws_layout(sh);
  uint8_t* p = static_cast<uint8_t*>(ws);
  return {reinterpret_cast<RowPlan*>(p + w.plan), reinterpret_cast<int*>(p + w.unit),
          reinterpret_cast<int*>(p + w.take)};
}

bool ws_ok(const kv_paged_shape& sh, const kv_paged_cache& c) {
  return aligned16(c.ws) && c.ws_bytes >= paged_ws_layout(sh).bytes;
}

// The rows of src -> dst lists: dst distinct, and no dst a src of its own cache except (in_place) its own entry's.
bool lists_ok(const int32_t* src, const int32_t* dst, int32_t n, bool same_cache, bool in_place) {
  if (!same_cache) return true;
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      if (dst[i] == src[j] && !(in_place && i == j)) return false;
  return true;
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" {

size_t kv_paged_page_bytes(const kv_paged_shape* shape) {
  return paged_shape_ok(shape) ? (size_t)page_geom(*shape).bytes : 0;
}

size_t kv_paged_ws_bytes(const kv_paged_shape* shape) {
  return paged_shape_ok(shape) ? paged_ws_layout(*shape).bytes : 0;
}

int kv_paged_rebuild(const kv_paged_shape* shape, const kv_paged_cache* cache, void* stream) {
  if (fault_injected("kv_paged_rebuild")) return KV_ERR_CUDA;
  if (!paged_shape_ok(shape) || !cache_ok(cache)) return KV_ERR_ARG;
  if (!ws_ok(*shape, *cache)) return KV_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const PageGeom g = page_geom(*shape);
  const PagedCache c = cache_of(*cache);
  const int rows = shape->n_seqs * shape->n_layers * shape->n_kv_heads;
  const PagedWs w = paged_ws_layout(*shape);
  if (cudaMemsetAsync(c.ref, 0, (size_t)g.n_pages * sizeof(int32_t), st) != cudaSuccess ||
      cudaMemsetAsync(static_cast<uint8_t*>(cache->ws) + w.arrived, 0, w.arrived_bytes, st) != cudaSuccess)
    return KV_ERR_CUDA;
  const int cap = sm_count() * 8;
  paged_count_kernel<<<rows < cap ? rows : cap, kRowThreads, 0, st>>>(g, rows, c);
  const int blocks = (g.n_pages + kRowThreads - 1) / kRowThreads;
  paged_bits_kernel<<<blocks < cap ? blocks : cap, kRowThreads, 0, st>>>(g.n_pages, c);
  return cuda_status(cudaGetLastError());
}

int kv_paged_append(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* seq, int32_t n_seq,
                    int32_t layer0, int32_t n_lay, const void* K, const void* V, int64_t n_src, int32_t n_each,
                    const int32_t* count, const int64_t* src_off, const int32_t* idx, const int64_t* idx_off,
                    void* stream) {
  if (fault_injected("kv_paged_append")) return KV_ERR_CUDA;
  if (!paged_shape_ok(shape) || !cache_ok(cache)) return KV_ERR_ARG;
  PlanArgs p = {};
  if (!make_rows(*shape, seq, n_seq, layer0, n_lay, true, &p.dst)) return KV_ERR_ARG;
  if (n_src < 0 || n_each < 0 || (n_src > 0 && (!aligned16(K) || !aligned16(V)))) return KV_ERR_ARG;
  if (count && !src_off) return KV_ERR_ARG;
  if (idx && (!src_off || !idx_off)) return KV_ERR_ARG;
  if (!list_ok(count) || !list_ok(src_off) || !list_ok(idx) || !list_ok(idx_off)) return KV_ERR_ARG;
  if (!ws_ok(*shape, *cache)) return KV_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Ws w = ws_of(*shape, cache->ws);
  p.g = page_geom(*shape);
  p.c = cache_of(*cache);
  p.count = count;
  p.n_each = n_each;
  p.plan = w.plan, p.unit = w.unit, p.take = w.take;
  int rc = launch(paged_plan_kernel<kAppend>, 1, kPlanThreads, st, p);
  if (rc) return rc;
  StoreArgs a = {p.g, p.dst, p.c, K, V, n_src, n_each, src_off, idx, idx_off, w.plan, w.unit, w.take};
  // a unit per warp while that leaves SMs idle; the batch's units are known on the device only, n_src bounds them
  const long long warps = n_src / kUnit + 2ll * p.dst.n_rows;
  const long long want = (warps + kMoveWarps - 1) / kMoveWarps;
  const int grid = (int)(want < INT_MAX ? want : INT_MAX);
  const bool f32 = shape->dtype == KV_F32;
  if (shape->head_dim == 64) return shape->quant_group == 32 ? store_as<64, 32>(f32, grid, a, st) : store_as<64, 64>(f32, grid, a, st);
  return shape->quant_group == 32   ? store_as<128, 32>(f32, grid, a, st)
         : shape->quant_group == 64 ? store_as<128, 64>(f32, grid, a, st)
                                    : store_as<128, 128>(f32, grid, a, st);
}

int kv_paged_load(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* seq, int32_t n_seq,
                  int32_t layer0, int32_t n_lay, const int64_t* out_off, int64_t n_out, void* K_out, void* V_out,
                  void* stream) {
  if (fault_injected("kv_paged_load")) return KV_ERR_CUDA;
  if (!paged_shape_ok(shape) || !cache_ok(cache)) return KV_ERR_ARG;
  LoadArgs a = {};
  if (!make_rows(*shape, seq, n_seq, layer0, n_lay, true, &a.rows)) return KV_ERR_ARG;
  if (!out_off || !list_ok(out_off) || n_out < 0 || !aligned16(K_out) || !aligned16(V_out))
    return KV_ERR_ARG;
  if (!ws_ok(*shape, *cache)) return KV_ERR_WORKSPACE;
  a.g = page_geom(*shape);
  a.c = cache_of(*cache);
  a.out_off = out_off, a.n_out = n_out, a.K = K_out, a.V = V_out;
  a.bits = shape->dtype == KV_F32 ? 0x4B000000u : 0x43004300u;
  const long long want = (n_out / kUnit + kMoveWarps) / kMoveWarps, cap = 4ll * sm_count();  // all resident
  const int grid = (int)(want < cap ? want : cap);
  const bool f32 = shape->dtype == KV_F32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->head_dim == 64) return shape->quant_group == 32 ? load_as<64, 32>(f32, grid, a, st) : load_as<64, 64>(f32, grid, a, st);
  return shape->quant_group == 32   ? load_as<128, 32>(f32, grid, a, st)
         : shape->quant_group == 64 ? load_as<128, 64>(f32, grid, a, st)
                                    : load_as<128, 128>(f32, grid, a, st);
}

int kv_paged_attn(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* seq, int32_t n_seq,
                  int32_t layer0, int32_t n_lay, int32_t n_q, const void* q, void* out, float* lse, void* stream) {
  if (fault_injected("kv_paged_attn")) return KV_ERR_CUDA;
  if (!paged_shape_ok(shape) || !cache_ok(cache)) return KV_ERR_ARG;
  SeqRows rows;
  if (!make_rows(*shape, seq, n_seq, layer0, n_lay, true, &rows)) return KV_ERR_ARG;
  if (n_q < 1 || n_q > KV_PAGED_MAX_QUERIES || n_q * shape->group > KV_PAGED_MAX_QUERIES) return KV_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || q == out) return KV_ERR_ARG;
  if (!list_ok(lse)) return KV_ERR_ARG;
  if (!ws_ok(*shape, *cache)) return KV_ERR_WORKSPACE;
  return launch_paged_attn(*shape, page_geom(*shape), rows, cache_of(*cache), static_cast<uint8_t*>(cache->ws), n_q, q,
                           out, lse, static_cast<cudaStream_t>(stream));
}

int kv_paged_fork(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* src, const int32_t* dst,
                  int32_t n, void* stream) {
  if (fault_injected("kv_paged_fork")) return KV_ERR_CUDA;
  if (!paged_shape_ok(shape) || !cache_ok(cache)) return KV_ERR_ARG;
  PlanArgs p = {};
  if (!make_rows(*shape, src, n, 0, shape->n_layers, false, &p.src) ||
      !make_rows(*shape, dst, n, 0, shape->n_layers, true, &p.dst) || !lists_ok(src, dst, n, true, false))
    return KV_ERR_ARG;
  if (!ws_ok(*shape, *cache)) return KV_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Ws w = ws_of(*shape, cache->ws);
  p.g = page_geom(*shape);
  p.c = cache_of(*cache);
  p.src_len = cache->len;
  p.src_max = shape->max_pages * shape->page_tokens;
  p.plan = w.plan, p.unit = w.unit, p.take = w.take;
  int rc = launch(paged_plan_kernel<kFork>, 1, kPlanThreads, st, p);
  if (rc) return rc;
  MoveArgs a = {p.g,           p.dst,            p.src,   p.c,     p.c.pages, p.c.table,
                shape->n_pages, shape->max_pages, nullptr, nullptr, w.plan,    w.unit,    w.take};
  return launch(paged_fork_kernel, p.dst.n_rows, kRowThreads, st, a);
}

// The address a kernel reaches pages at: device or managed memory as is, pinned host memory at its device mapping.
static uint8_t* pages_address(void* p) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  if (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) return static_cast<uint8_t*>(p);
  if (at.type == cudaMemoryTypeHost && at.devicePointer) return static_cast<uint8_t*>(at.devicePointer);
  return nullptr;
}

int kv_paged_copy(const kv_paged_shape* src_shape, const kv_paged_cache* src_cache, const int32_t* src,
                  const kv_paged_shape* dst_shape, const kv_paged_cache* dst_cache, const int32_t* dst, int32_t n,
                  void* stream) {
  if (fault_injected("kv_paged_copy")) return KV_ERR_CUDA;
  if (!paged_shape_ok(src_shape) || !paged_shape_ok(dst_shape) || !cache_ok(src_cache) || !cache_ok(dst_cache))
    return KV_ERR_ARG;
  if (src_shape->n_layers != dst_shape->n_layers || src_shape->n_kv_heads != dst_shape->n_kv_heads ||
      src_shape->head_dim != dst_shape->head_dim || src_shape->quant_group != dst_shape->quant_group ||
      src_shape->page_tokens != dst_shape->page_tokens)
    return KV_ERR_ARG;
  PlanArgs p = {};
  if (!make_rows(*src_shape, src, n, 0, src_shape->n_layers, false, &p.src) ||
      !make_rows(*dst_shape, dst, n, 0, dst_shape->n_layers, true, &p.dst) ||
      !lists_ok(src, dst, n, src_cache->table == dst_cache->table, false))
    return KV_ERR_ARG;
  if (!ws_ok(*dst_shape, *dst_cache)) return KV_ERR_WORKSPACE;
  uint8_t* sp = pages_address(src_cache->pages);
  uint8_t* dp = pages_address(dst_cache->pages);
  if (!sp || !dp) return KV_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Ws w = ws_of(*dst_shape, dst_cache->ws);
  p.g = page_geom(*dst_shape);
  p.c = cache_of(*dst_cache);
  p.c.pages = dp;
  p.src_len = src_cache->len;
  p.src_max = src_shape->max_pages * src_shape->page_tokens;
  p.plan = w.plan, p.unit = w.unit, p.take = w.take;
  int rc = launch(paged_plan_kernel<kCopy>, 1, kPlanThreads, st, p);
  if (rc) return rc;
  MoveArgs a = {p.g,   p.dst, p.src,  p.c,    sp, src_cache->table, src_shape->n_pages, src_shape->max_pages, nullptr,
                nullptr, w.plan, w.unit, w.take};
  // enough CTAs to fill the SMs when rows are few
  const int want = 8 * sm_count() / p.dst.n_rows + 1;
  const int slices = want < dst_shape->max_pages ? want : dst_shape->max_pages;
  return launch(paged_copy_kernel, dim3(p.dst.n_rows, slices), kRowThreads, st, a);
}

int kv_paged_compact(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* src,
                     const int32_t* dst, int32_t n, const int32_t* idx, const int64_t* idx_off,
                     const int32_t* count, void* stream) {
  if (fault_injected("kv_paged_compact")) return KV_ERR_CUDA;
  if (!paged_shape_ok(shape) || !cache_ok(cache)) return KV_ERR_ARG;
  PlanArgs p = {};
  if (!make_rows(*shape, src, n, 0, shape->n_layers, false, &p.src) ||
      !make_rows(*shape, dst, n, 0, shape->n_layers, true, &p.dst) || !lists_ok(src, dst, n, true, true))
    return KV_ERR_ARG;
  if (!idx || !idx_off || !count || !list_ok(idx) || !list_ok(idx_off) || !list_ok(count)) return KV_ERR_ARG;
  if (!ws_ok(*shape, *cache)) return KV_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Ws w = ws_of(*shape, cache->ws);
  p.g = page_geom(*shape);
  p.c = cache_of(*cache);
  p.src_len = cache->len;
  p.src_max = shape->max_pages * shape->page_tokens;
  p.count = count;
  p.plan = w.plan, p.unit = w.unit, p.take = w.take;
  int rc = launch(paged_plan_kernel<kCompact>, 1, kPlanThreads, st, p);
  if (rc) return rc;
  MoveArgs a = {p.g,           p.dst,            p.src, p.c,     p.c.pages, p.c.table,
                shape->n_pages, shape->max_pages, idx,   idx_off, w.plan,    w.unit,    w.take};
  const long long want = ((long long)shape->n_pages * shape->page_tokens / kUnit + kMoveWarps - 1) / kMoveWarps;
  const long long cap = 8ll * sm_count();
  rc = launch(paged_compact_kernel, (int)(want < cap ? want : cap), kMoveWarps * 32, st, a);
  if (rc) return rc;
  return launch(paged_commit_kernel, p.dst.n_rows, kRowThreads, st, a);
}

int kv_paged_free(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* seq, int32_t n_seq,
                  void* stream) {
  if (fault_injected("kv_paged_free")) return KV_ERR_CUDA;
  if (!paged_shape_ok(shape) || !cache_ok(cache)) return KV_ERR_ARG;
  SeqRows rows;
  if (!make_rows(*shape, seq, n_seq, 0, shape->n_layers, true, &rows)) return KV_ERR_ARG;
  return launch(paged_free_kernel, rows.n_rows, kRowThreads, static_cast<cudaStream_t>(stream), page_geom(*shape),
                rows, cache_of(*cache));
}

}  // extern "C"

// Definitions shared by the paged 4-bit cache's kernels (paged.cu: storing,
// reading and moving tokens and pages; paged_attn.cu: attention): the shape
// of a page, the rows a call names, the layout of the workspace, and launches.
#pragma once

#include <atomic>

#include "../../include/kvcomp_paged.h"
#include "internal.h"

namespace kvc {

// Byte offsets within a page: K codes at 0, V codes at v, K scales at ks, V scales at vs.
struct PageGeom {
  int P, log_p;  // tokens per page
  int d, G, qg;
  int v, ks, vs, bytes;
  int n_pages, max_pages;
};

// The table rows of a call: call row i is row `first + i % per_seq` of sequence seq[i / per_seq].
struct SeqRows {
  int n_seq;
  int per_seq;    // call rows of a sequence
  int first;      // layer0 * n_kv_heads
  int table_rps;  // table rows of a sequence
  int n_rows;     // n_seq * per_seq
  int seq[KV_MAX_SEQ];
};
__device__ __forceinline__ int table_row(const SeqRows& r, int i) {
  const int s = i / r.per_seq;
  return r.seq[s] * r.table_rps + r.first + (i - s * r.per_seq);
}

struct PagedCache {
  uint8_t* pages;
  int32_t* table;
  int32_t* len;
  int32_t* ref;
  uint32_t* free_bits;
  int32_t* status;
};

// What the plan kernel decided for a call row.
struct RowPlan {
  int take;   // rank of its first new page in the list of taken pages
  int fresh;  // index of its first new page in the row's list; -1: the row is left as it was
  int old;    // tokens before the call (append: of the row; fork, copy, compact: of the source)
  int n;      // tokens to store, move or share
};

// Workspace: the attention's counters (0 between calls) and partials, plans
// and unit prefix of the call rows, the pages taken.
struct PagedWs {
  size_t arrived, arrived_bytes, part, plan, unit, take, bytes;
};
constexpr int kUnit = 16;            // tokens per unit of the storing and moving kernels
constexpr int kAttnRows = 1024;      // call rows per attention launch
constexpr int kAttnQ = 16;           // query rows per attention CTA, at most
constexpr int kAttnCtasPerSm = 3;    // at most
PagedWs paged_ws_layout(const kv_paged_shape& sh);
PageGeom page_geom(const kv_paged_shape& sh);
bool paged_shape_ok(const kv_paged_shape* sh);

// (x & mask) | bits in one instruction: it takes one constant, so the other comes in a register.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "n"(MASK), "r"(bits));
  return r;
}

// Launch whose set-up overlaps the previous kernel's tail. Every paged kernel waits for that kernel before it touches
// memory, and reads with plain loads (the read-only path may not see what a kernel that was still running wrote).
template <class... P, class... A>
int launch_smem(void (*k)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, k, P(args)...));
}
template <class... P, class... A>
int launch(void (*k)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  return launch_smem(k, grid, threads, 0, st, args...);
}

// Lets kernel k take `bytes` of shared memory on the current device; `ready` holds the devices where it may already.
template <class... P>
int allow_smem(void (*k)(P...), int bytes, std::atomic<unsigned long long>& ready) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KV_ERR_CUDA;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (ready.load(std::memory_order_relaxed) & bit) return KV_OK;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return KV_ERR_CUDA;
  ready.fetch_or(bit, std::memory_order_relaxed);
  return KV_OK;
}

int launch_paged_attn(const kv_paged_shape& sh, const PageGeom& g, const SeqRows& rows, const PagedCache& c,
                      uint8_t* ws, int n_q, const void* q, void* out, float* lse, cudaStream_t st);

}  // namespace kvc

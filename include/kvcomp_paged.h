/*
 * kvcomp_paged.h — a paged KV cache held in 4 bits: storing kept tokens into
 * it, attention over it, and copying, forking, compacting and freeing its
 * pages. (No counterpart on the pages beyond the remark that quantising the
 * kept cache to 4 bits is future work, AudioKV blog §6; the pages of one row
 * follow from the per-head budgets of AudioKV blog §3.1, which give every
 * (sequence, layer, KV head) a length of its own.)
 *
 * Conventions are those of kvcomp.h and kvcomp_next.h: caller-owned device buffers, nothing
 * allocated, nothing synchronised, every call asynchronous on `stream`, a
 * status returned before anything is launched, device-detected problems OR-ed
 * into a status word. Every call may be captured into a CUDA graph.
 *
 * Rows. A cache has room for n_seqs sequences of n_layers x n_kv_heads rows:
 * table row = (sequence * n_layers + layer) * n_kv_heads + head. Each row has
 * its own length len[row] and its own list of pages, table[row][0 ..
 * ceil(len / page_tokens)): page j holds tokens [j P, (j + 1) P) of the row, P =
 * page_tokens. Entries behind that are not read and keep what they hold.
 * A call names its sequences by a host list seq[n_seq] (n_seq <= KV_MAX_SEQ,
 * no sequence twice) and a range of layers [layer0, layer0 + n_lay); its call
 * rows are (s * n_lay + layer - layer0) * n_kv_heads + head in the order of
 * the list, and per-row arguments hold one entry for each of them.
 *
 * Pages. ref[p] counts the rows whose list holds page p; free_bits has bit p
 * of word p / 32 set while it is 0. A page that is filled in part belongs to
 * one row only. New pages are the lowest-numbered free ones, handed out in
 * call-row order, then page order. A call whose rows need more pages than are
 * free serves rows in order while they last: a row whose pages do not fit is
 * left as it was and sets KV_DEV_PAGES.
 *
 * Quantisation, per token of K or V and group of quant_group channels:
 *   m = bf16(min x),  s = bf16(f32((max x - m) / 15)) (0 unless max x > m),
 *   c = clamp(rint((x - m) / s), 0, 15) (halves to even, the quotient exact;
 *   0 where s = 0);  the value held is m + c s.
 * A group with a NaN or an infinity, or whose smallest value rounds to one, holds NaN.
 *
 * Page layout (kv_paged_page_bytes() bytes, G = head_dim / quant_group):
 *   K codes [P][d / 2 bytes], V codes [P][d / 2 bytes], K scales [P][G],
 *   V scales [P][G]; a scale is s (bf16, low half) and m (bf16, high half).
 *   K codes of a token: 32-bit words [4][d / 32]; word (t, w) holds dims
 *   32 w + 8 t + n in bits 4 n, n = 0..7.
 *   V codes of a token: 16-bit words [8][d / 32]; word (p, h) holds dims
 *   32 h + 4 g + n in bits 4 n, n = 0..3, with g = p, or p ^ 4 where bit 1 of
 *   the token's place in its page is set.
 *
 * Order. Calls on one cache must be ordered: one stream, or events between
 * streams. kv_paged_attn and kv_paged_load only read the cache but share its
 * workspace with every other call; to run them beside others give them a
 * kv_paged_cache that names a workspace of its own.
 */
#ifndef KVCOMP_PAGED_H
#define KVCOMP_PAGED_H

#include "kvcomp_next.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KV_PAGED_MAX_ROWS (1 << 20)    /* n_seqs * n_layers * n_kv_heads           */
#define KV_PAGED_MAX_PAGES (1 << 24)   /* n_pages                                  */
#define KV_PAGED_MAX_TOKENS (1 << 26)  /* max_pages * page_tokens: tokens of a row    */
#define KV_PAGED_MAX_QUERIES 64        /* n_q * group of kv_paged_attn             */

/* Device status bits of the paged calls, beside those of kvcomp.h and kvcomp_next.h:
 * KV_DEV_CAPACITY (a row's list would pass max_pages), KV_DEV_BOUNDS (a page
 * number outside the pool, a length outside the table) and KV_DEV_RANGE (
 * a source row or kept position that does not exist; stored as zeros). */
#define KV_DEV_PAGES 0x20 /* the pool has no free page for a row               */
#define KV_DEV_BUSY 0x40  /* a destination row that already holds tokens       */

typedef struct {
  int32_t n_seqs;      /* sequences the cache has room for                    */
  int32_t n_layers;    /* layers per sequence                                 */
  int32_t n_kv_heads;  /* H: KV heads per layer                               */
  int32_t group;       /* g: query heads per KV head, 1..16                   */
  int32_t head_dim;    /* d: 64 or 128                                        */
  int32_t dtype;       /* type of q, K, V and outputs: KV_BF16 or KV_F32      */
  int32_t n_pages;     /* pages of the pool                                   */
  int32_t max_pages;   /* pages of a row, at most (width of the table)        */
  int32_t quant_group; /* channels that share a scale: 32, 64 or 128, <= d    */
  int32_t page_tokens; /* P: 16, 32, 64 or 128                                */
} kv_paged_shape;

typedef struct {
  void* pages;         /* [n_pages][kv_paged_page_bytes()], 16-byte aligned   */
  int32_t* table;      /* [n_seqs * n_layers * n_kv_heads][max_pages]         */
  int32_t* len;        /* [n_seqs * n_layers * n_kv_heads]                    */
  int32_t* ref;        /* [n_pages]                                           */
  uint32_t* free_bits; /* [ceil(n_pages / 32)]                                */
  int32_t* status;     /* device status word (KV_DEV_* bits are OR-ed in)     */
  void* ws;            /* kv_paged_ws_bytes() bytes, prepared by              */
  size_t ws_bytes;     /*   kv_paged_rebuild (or zeroed) before its first use */
} kv_paged_cache;

/* Bytes of a page, or 0 on a bad shape. */
size_t kv_paged_page_bytes(const kv_paged_shape* shape);

/* Bytes of workspace that any call on this shape needs on the current device, or 0 on a bad shape. */
size_t kv_paged_ws_bytes(const kv_paged_shape* shape);

/*
 * kv_paged_rebuild — ref and free_bits from table and len, and the workspace:
 * what a cache needs before its first call (with len = 0 it is empty) and after
 * its state was loaded from elsewhere. Page numbers outside the pool set KV_DEV_BOUNDS.
 * Errors: KV_ERR_ARG, KV_ERR_WORKSPACE, KV_ERR_CUDA.
 */
int kv_paged_rebuild(const kv_paged_shape* shape, const kv_paged_cache* cache, void* stream);

/*
 * kv_paged_append — quantises tokens and stores them behind each row's last.
 *   K, V    : device, [n_src][d] dtype (both the same rows; not looked at where n_src = 0).
 *   count   : device int32 [call rows], tokens of each row (0 or more; a
 *             negative count is 0), or NULL: n_each tokens a row.
 *   src_off : device int64 [call rows], the source row that a row's positions
 *             count from, or NULL: i * n_each for call row i (count NULL only).
 *   idx     : device int32, or NULL. Token t of call row i is source row
 *             src_off[i] + idx[idx_off[i] + t], without idx src_off[i] + t.
 *   idx_off : device int64 [call rows] (more entries are not read), with idx.
 *   idx holds every entry that a row's idx_off and count reach; the call cannot
 *   check that. Lists are aligned to their type (KV_ERR_ARG).
 *   With count = b, idx and idx_off = slot_off of kv_select_gather (or of
 *   kv_select) and src_off = the rows' key offsets this stores the kept tokens
 *   of a batch without the compacted copy in between.
 * A row whose list would pass max_pages is left as it was (KV_DEV_CAPACITY).
 * Errors: KV_ERR_ARG, KV_ERR_WORKSPACE, KV_ERR_CUDA.
 */
int kv_paged_append(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* seq, int32_t n_seq,
                    int32_t layer0, int32_t n_lay, const void* K, const void* V, int64_t n_src, int32_t n_each,
                    const int32_t* count, const int64_t* src_off, const int32_t* idx, const int64_t* idx_off,
                    void* stream);

/*
 * kv_paged_load — the values of the rows' tokens, rounded to dtype:
 *   token t of call row i goes to row out_off[i] + t of K_out and V_out, for
 *   t < min(len, out_off[i + 1] - out_off[i]); other rows are left as they are.
 *   out_off : device int64 [call rows + 1], ascending from 0 or more, the last
 *             at most n_out (rows of K_out and V_out); what passes n_out is
 *             not written and sets KV_DEV_RANGE.
 * Errors: KV_ERR_ARG, KV_ERR_WORKSPACE, KV_ERR_CUDA.
 */
int kv_paged_load(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* seq, int32_t n_seq,
                  int32_t layer0, int32_t n_lay, const int64_t* out_off, int64_t n_out, void* K_out, void* V_out,
                  void* stream);

/*
 * kv_paged_attn — attention of n_q query tokens of every row over its cache,
 * their own tokens appended before the call:
 *   query token t of a row sees keys 0 .. len - n_q + t;
 *   out = softmax(q K^T / sqrt(d)) V over them,  lse = log sum exp(q K^T / sqrt(d))
 *   with K and V the values held. A query that sees no key gives out = 0 and
 *   lse = -infinity. Sums are float32's: a logit is off by at most
 *   (d + 16) 2^-23 sum_c |q_c| (16 s_c + |m_c|) / sqrt d (s and m the step and
 *   base that channel c is held with). KV_BF16 rounds a key's weight times its V
 *   step to fp16, 2^-11 of it (to 16 bits where V steps of a row lie far apart),
 *   KV_F32 to 24 bits; channels, tokens and queries of any size beside each other
 *   cost one another nothing.
 *   q, out : device, [call rows][n_q][g][d] dtype (out may not overlap q).
 *   lse    : device float32 [call rows][n_q][g], or NULL.
 *   n_q * group <= KV_PAGED_MAX_QUERIES. Queries are finite, and queries and values held below
 *   2^100 in magnitude (sums over larger ones may pass float32's range); a query that is not
 *   spoils its own output only, a NaN held the outputs of the queries that see it.
 * Results do not depend on where the pages lie; repeated calls give the same bits.
 * Errors: KV_ERR_ARG, KV_ERR_WORKSPACE, KV_ERR_CUDA.
 */
int kv_paged_attn(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* seq, int32_t n_seq,
                  int32_t layer0, int32_t n_lay, int32_t n_q, const void* q, void* out, float* lse, void* stream);

/*
 * kv_paged_fork — every layer of sequences dst[i] becomes a second holder of
 * src[i]'s tokens: full pages are shared, the page filled in part is copied.
 * src may name a sequence more than once; no dst twice and none that is a src.
 * A dst row that holds tokens is left as it was (KV_DEV_BUSY).
 * Errors: KV_ERR_ARG, KV_ERR_WORKSPACE, KV_ERR_CUDA.
 */
int kv_paged_fork(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* src, const int32_t* dst,
                  int32_t n, void* stream);

/*
 * kv_paged_copy — copies every page of sequences src[i] of one cache into
 * pages of dst[i] of another (or of the same cache), shared with no one. Both
 * shapes agree in n_layers, n_kv_heads, head_dim, quant_group and page_tokens.
 * `pages` of either cache may be pinned host memory here (the copy then
 * crosses the host link); its other arrays are device memory as always.
 * No dst twice; within one cache (the same table) none that is a src. Rows
 * are refused as by kv_paged_fork and, past dst's max_pages, KV_DEV_CAPACITY;
 * status bits go to dst's word.
 * Errors: KV_ERR_ARG, KV_ERR_WORKSPACE (dst's), KV_ERR_CUDA.
 */
int kv_paged_copy(const kv_paged_shape* src_shape, const kv_paged_cache* src_cache, const int32_t* src,
                  const kv_paged_shape* dst_shape, const kv_paged_cache* dst_cache, const int32_t* dst, int32_t n,
                  void* stream);

/*
 * kv_paged_compact — keeps the listed tokens: row r of dst[i] holds tokens
 * idx[idx_off[r] + t], t < count[r], of the same row of src[i], in new pages,
 * codes and scales unchanged. dst[i] is src[i] (replaced in place: its former
 * pages are given up afterwards, so the new ones have to be free before) or a
 * sequence whose rows are empty (KV_DEV_BUSY otherwise) and which is no src.
 * src may name a sequence more than once, but not one that is replaced.
 *   idx     : device int32 positions below the row's length, in any order (one
 *             that is not below it is stored as zeros, KV_DEV_RANGE).
 *   idx_off : device int64 [n * n_layers * n_kv_heads] (more are not read).
 *   count   : device int32 [n * n_layers * n_kv_heads]; a negative count is 0.
 *   As for kv_paged_append, idx holds every entry that is reached, and lists are
 *   aligned to their type.
 * A row whose list would pass max_pages is left as it was (KV_DEV_CAPACITY).
 * Errors: KV_ERR_ARG, KV_ERR_WORKSPACE, KV_ERR_CUDA.
 */
int kv_paged_compact(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* src,
                     const int32_t* dst, int32_t n, const int32_t* idx, const int64_t* idx_off,
                     const int32_t* count, void* stream);

/*
 * kv_paged_free — the sequences' rows become empty; pages that no other row
 * holds are free again. Errors: KV_ERR_ARG, KV_ERR_CUDA.
 */
int kv_paged_free(const kv_paged_shape* shape, const kv_paged_cache* cache, const int32_t* seq, int32_t n_seq,
                  void* stream);

/*
 * kv_select — the selection of kv_select_gather without the gather: idx gets
 * the kept positions of every row, for kv_paged_append to store from K and V.
 * Arguments as kv_select_gather. Errors: KV_ERR_ARG, KV_ERR_UNSUPPORTED_L, KV_ERR_CUDA.
 */
int kv_select(const kv_shape* shape, const int32_t* L, int32_t n_seq, const float* s_hat, const int32_t* b,
              const int64_t* slot_off, int32_t* idx, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVCOMP_PAGED_H */

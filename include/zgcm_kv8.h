/*
 * zgcm_kv8.h — C ABI of a KV cache held in 8 bits by blocks of 64 tokens, and of the decode
 * attention over it (sm_100a): filling it from prompts and single tokens, the gated attention
 * of one new token per sequence, and the choice of the blocks that a long context's attention
 * reads.
 *
 * The growing caches of the global layers are what a decode step reads (ZGCM-1 KV design,
 * ZGCM-1 summary section "前置知识"; 32 GiB at 256K tokens for full attention, shibing624
 * review section "架构"); 8-bit codes halve them, selected blocks read a fraction of them.
 *
 * Blocks.  Block j of a sequence is its positions 64 j .. 64 j + 63.  A block that is whole
 * lives in a page as codes: for each KV head and each of keys and values
 *      scale = max(amax * (1/M), 2^-126),  code = round(x / scale)    (nearest, ties to even)
 * with amax = max |x| over the head's 64 x 128 values, M = 448 for ZGCM_E4M3 and 127 for
 * ZGCM_INT8, all in fp32, 1/M rounded too; a code stands for code * scale.  If amax is not finite the scale is
 * NaN and the codes 0: the block then reads as NaN for that head.  Beside the codes the page
 * holds the mean of its 64 keys.  The block of a sequence's newest token is also held as it was
 * given, in 16 bits, in the sequence's tail: a block is coded once, when its last token
 * arrives, from the 16-bit values, so what a cache holds does not depend on how the tokens
 * were split over calls.
 *
 * Tables.  Block j of sequence b is in page table[b][j mod n_blocks].  With n_blocks at least
 * the longest sequence's number of blocks the cache grows; with ceil((window-1)/64) + 1 blocks
 * it is a sliding layer's ring.  A call that needs a block which the ring has overwritten, or
 * whose page number is outside 0 .. n_pages-1, answers NaN for the rows concerned and reads
 * and writes nothing there.  Sequences may share pages of whole blocks that none of them will
 * write again (a common prefix).  Pages written by one call must be distinct.
 *
 * Keys and queries are taken prepared (normalised and rotated: zgcm_qkrope.h), in key_type;
 * values, gates and outputs are bf16.
 *
 * Positions are device memory (pos int32 [n_seq]), so that a captured graph follows them.
 * pos[b] < 0 marks an idle sequence: its cache and table are not touched.
 *
 * Errors and streams as in zgcm_attn.h.  Pointers 16-byte aligned.  D == 128, Hq % Hkv == 0.
 */
#ifndef ZGCM_KV8_H
#define ZGCM_KV8_H

#include "zgcm_qkrope.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZGCM_KV8_BLOCK 64

typedef enum { ZGCM_E4M3 = 0, ZGCM_INT8 = 1 } zgcm_code_type;

typedef struct {
    void* k_codes;     /* [n_pages, Hkv, 64, D], 1 byte each */
    void* v_codes;     /* [n_pages, Hkv, 64, D] */
    float* k_scale;    /* [n_pages, Hkv] */
    float* v_scale;    /* [n_pages, Hkv] */
    void* k_mean;      /* [n_pages, Hkv, D], key_type */
    void* k_tail;      /* [n_seq, Hkv, 64, D], key_type */
    void* v_tail;      /* [n_seq, Hkv, 64, D], bf16 */
    const int* table;  /* [n_seq, n_blocks] page numbers */
    int n_seq, n_blocks, n_pages, Hkv, D;
    int code_type;     /* zgcm_code_type */
    int key_type;      /* ZGCM_BF16 or ZGCM_FP16 */
} zgcm_kv8_cache;

/*
 * Append tokens: k, v [n_seq, N, Hkv, D] (element (b, i, h, d) at b * b_stride + i * t_stride
 * + h * h_stride + d; strides multiples of 8), the first of them at position pos[b], count[b]
 * of them (count NULL: N each; values outside 0 .. N are taken as the nearer bound).  The
 * cache must hold positions 0 .. pos[b]-1 of the sequence already.  Rows i >= count[b] are not
 * read.  Blocks that the call completes are coded, except those that the ring overwrites
 * within the same call; the newest block is written to the tail, whose rows past the newest
 * token keep what they hold.  A block whose page number is bad is not stored.
 *
 * Rewinding (a rejected draft, an answer given anew): pos[b] may be any position of the block of
 * the last token appended, or the first position (a multiple of 64) of an earlier block; the
 * tokens from there on are then those of this call.  Not a position inside an earlier block: that
 * block's first tokens would be taken from the tail, which has held a later block since, and the
 * call cannot know; append it from its first position.  A ring that has stored later blocks has lost
 * those that they replaced: a sequence can go back by as many blocks as n_blocks exceeds the
 * ceil((window-1)/64) + 1 that its window touches.
 */
int zgcm_kv8_append(const zgcm_kv8_cache* cache, const void* k, long long k_b_stride, long long k_t_stride,
                    long long k_h_stride, const void* v, long long v_b_stride, long long v_t_stride,
                    long long v_h_stride, const int* pos, const int* count, int N, void* cuda_stream);

/*
 * Decode attention of one token per sequence at position p = pos[b], the newest one appended:
 *      out = sigmoid(g) * softmax_j(scale q . k_j) v_j  over j = max(0, p-window+1) .. p,
 *      lse = log sum_j exp(scale q . k_j)
 * with k_j, v_j of p's own block floor(p/64) as in the tail and of earlier blocks as their
 * codes stand for.  blocks (may be NULL): int32 [n_seq, Hkv, n_list], the earlier blocks to
 * read, ascending, for example from zgcm_kv8_select; an entry that is negative, not below p's own
 * block, wholly before the window or not above the entry before it is passed over.  (The entry directly before is
 * all that is looked at: a list that is not ascending may bring a block in twice.)  The own block is always read.
 * q [n_seq, Hq, D] key_type; g [n_seq, Hq, D] bf16, or NULL for no gate (out = the softmax's
 * mean); out bf16 [n_seq, Hq, D]; lse fp32 [n_seq, Hq].  Idle sequences: out 0, lse -inf.
 * A window that reaches further back than n_blocks blocks (the own one among them): NaN.
 * Probabilities enter their products with 22 bits or more; scores, sums and out are fp32 and out is rounded once.  A value of the
 * own block that is not finite makes out not finite in its dim.  v_scale times 2^-14 is fp32: blocks of values below 2^-103 lose bits.
 * workspace: zgcm_attn_decode_kv8_workspace_size bytes (n_list < 0: no list), 16-byte aligned, contents on
 * entry irrelevant, not used by a concurrent call.  0, and workspace may be NULL, where no sequence can have many blocks to
 * read, and for arguments that zgcm_attn_decode_kv8 rejects; positions do not matter.
 */
size_t zgcm_attn_decode_kv8_workspace_size(const zgcm_kv8_cache* cache, int Hq, int window, int n_list);

int zgcm_attn_decode_kv8(const zgcm_kv8_cache* cache, const void* q, const void* g, const int* pos, const int* blocks,
                         int n_list, int Hq, int window, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* cuda_stream);

/*
 * Choose blocks: for each sequence at position p = pos[b] and each KV head, n_select of the
 * blocks before p's own that the window reaches (the candidates):
 *      score_j = max over the head's queries of q . k_mean_j      (fp64 sums)
 * The first n_first and the last n_last candidates always come first, then the highest scores;
 * equal scores go to the lowest block, a score with a NaN counts as -inf.  Out: blocks int32
 * [n_seq, Hkv, n_select], ascending, -1 behind the last where there are fewer candidates (all
 * -1 for an idle sequence, and where the window reaches an overwritten block).
 * 0 <= n_first, n_last; n_first + n_last <= n_select; n_select >= 1; n_blocks <= 16384
 * (1M tokens; ZGCM_ERR_UNSUPPORTED above).
 */
int zgcm_kv8_select(const zgcm_kv8_cache* cache, const void* q, const int* pos, int Hq, int window, int n_select,
                    int n_first, int n_last, int* blocks, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* ZGCM_KV8_H */

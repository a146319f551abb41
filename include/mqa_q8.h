/*
 * libmqa, 8-bit K/V caches: the cache's rows quantised as they are written,
 * read back, and attended to by single-token queries — each sequence over its
 * own rows, or a whole batch behind one shared prefix.
 *
 * The attention is that of mqa.h (mqa_decode): the velog paper review of
 * "Fast Transformer Decoding", §3 MultiquerySelfAttentionIncremental, with the
 * GQA blog's grouping (query head i reads K/V head i / (h/g)).  The pages keep
 * the cache in the model's type; here a row of one K/V head, x[0..d), is kept
 * as d e4m3 codes and one exponent byte E:
 *
 *   x[c] = code[c] * s,  s = the fp32 number with exponent field E and
 *                        mantissa 0: 2^(E-127), 0 for E = 0, +inf for E = 255
 *
 *   codes      device uint8 [b, m_max, g, d]   e4m3 (no infinities; 0x7f/0xff
 *                                              are NaN; largest 448)
 *   exponents  device uint8 [b, g, m_max]
 *
 * The library writes E in [1, 254]; rows that are attended to must not hold
 * E = 255.  A power of two costs e4m3 no precision (it is a floating format),
 * makes code * s exact in bf16 and fp32, and makes quantising what was read
 * back keep every value (a row whose largest value was rounded down to 224 s
 * gets twice the codes at half the scale).  The exponents of one head lie in
 * row order, so a tile's are one short run.
 *
 * Conventions are those of mqa.h: caller-owned device pointers on the current
 * device, 16-byte aligned except the exponent arrays (any alignment) and the
 * packed rows of mqa_q8_append and mqa_q8_read (32-byte aligned), not aliased;
 * dense row-major tensors; asynchronous on `stream`; arguments checked before
 * any launch; no allocation, no state between calls, no exceptions; device-read
 * values are clamped or skipped and reported in *status_flags (NULL to ignore).
 */
#ifndef LIBMQA_MQA_Q8_H
#define LIBMQA_MQA_Q8_H

#include "mqa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mqa_q8_append — quantise new rows and write them into the cache.
 *
 *   k_codes, k_exps  device [b, m_max, g, d_k] and [b, g, m_max], written at
 *   v_codes, v_exps  device [b, m_max, g, d_v] and [b, g, m_max]   new rows only
 *   k_new    device [total, g, d_k]  read     (dtype: fp32 or bf16)
 *   v_new    device [total, g, d_v]  read
 *   pos      device int32 [b]        cache row of a sequence's first new row
 *   cu_new   device int32 [b+1] or NULL: new rows cu_new[s] .. cu_new[s+1]-1
 *            belong to sequence s (non-decreasing from 0); NULL: one row per
 *            sequence, total = b
 *
 * A row's exponent is the smallest s = 2^(E-127), E in [1, 254], with
 * |x| <= 448 s for every finite x of the row (E = 1 for a row of zeros); its
 * codes are x / s rounded to e4m3, nearest with ties to even.  Infinities
 * become +-448 s, NaN stays NaN.  (A value that rounds up past the largest
 * number of its type reads back as infinity.)
 * Rows that would land outside [0, m_max) are skipped and set
 * MQA_FLAG_POS_SKIPPED; rows of k_new that belong to no sequence are ignored.
 * b = 0 or total = 0 is a no-op.  d_k and d_v in {16, 32, 64, 128, 256}
 * (MQA_ERR_UNSUPPORTED otherwise).
 */
MQA_API mqa_status_t mqa_q8_append(void* k_codes, uint8_t* k_exps, void* v_codes, uint8_t* v_exps, const void* k_new,
                                   const void* v_new, const int32_t* pos, const int32_t* cu_new, int b, int total,
                                   int m_max, int g, int d_k, int d_v, mqa_dtype_t dtype, int32_t* status_flags,
                                   cudaStream_t stream);

/*
 * mqa_q8_read — the values of cached rows, packed.
 *
 *   k_out    device [total, g, d_k]  written  (dtype: fp32 or bf16)
 *   v_out    device [total, g, d_v]  written
 *   start    device int32 [b] or NULL (all 0): first cache row read of each
 *            sequence
 *   cu_rows  device int32 [b+1]: packed rows cu_rows[s] .. cu_rows[s+1]-1 are
 *            cache rows start[s], start[s]+1, ... of sequence s
 *
 * Exact in both types (bf16 keeps more bits than a code has), but for values
 * outside the type's range.  Packed rows whose cache row lies outside
 * [0, m_max) are left as they were and set MQA_FLAG_POS_SKIPPED; so are,
 * without a flag, rows that belong to no sequence.  Sizes and errors as for
 * mqa_q8_append.
 */
MQA_API mqa_status_t mqa_q8_read(void* k_out, void* v_out, const void* k_codes, const uint8_t* k_exps,
                                 const void* v_codes, const uint8_t* v_exps, const int32_t* start,
                                 const int32_t* cu_rows, int b, int total, int m_max, int g, int d_k, int d_v,
                                 mqa_dtype_t dtype, int32_t* status_flags, cudaStream_t stream);

/*
 * mqa_q8_decode — mqa_decode_ex over an 8-bit cache.
 *
 *   o        device [b, h, d_v]   written (dtype of q: fp32 or bf16)
 *   q        device [b, h, d_k]
 *   lens     device int32 [b]     as for mqa_decode (clamped to [0, m_max];
 *                                 0 gives a zero row)
 *   workspace  device, mqa_q8_decode_workspace_size(b, h, g, d_v) bytes,
 *              256-byte aligned, contents on entry do not matter; calls that
 *              share one must be ordered on one stream
 *   opts     path, CTA count and local window, as for mqa_decode_ex, or NULL
 *
 * Rows at or past lens[b], and rows before the window, never count, whatever
 * codes and exponents they hold.  Statistics and sums are fp32.  On the
 * tensor-core path a row's weight is off by at most 2^-9 + 2^-11 of itself and
 * less than a step of 2^-17 of the largest p_t s_t (weight times value scale),
 * up or down as often as its size says; a query's elements by at most 2^-17 of
 * its largest.  There the value scales of one K/V head's rows, rows of zeros aside,
 * are at most 2^100 apart.
 * Paths: the tensor-core path takes bf16 with d_k = d_v = 128 and h/g <= 64,
 * and is then the automatic choice; the CUDA-core path takes both types with
 * d_k, d_v in {32, 64, 128} and h/g * d_k, h/g * d_v <= 4096.
 * MQA_ERR_UNSUPPORTED for other shapes.  q holding an infinity or NaN gives a
 * NaN output for that head.
 */
MQA_API size_t mqa_q8_decode_workspace_size(int b, int h, int g, int d_v);
MQA_API mqa_status_t mqa_q8_decode(void* o, const void* q, const void* k_codes, const uint8_t* k_exps,
                                   const void* v_codes, const uint8_t* v_exps, const int32_t* lens, int b, int h, int g,
                                   int m_max, int d_k, int d_v, float scale, mqa_dtype_t dtype, void* workspace,
                                   size_t workspace_bytes, int32_t* status_flags, const mqa_decode_opts_t* opts,
                                   cudaStream_t stream);

/*
 * mqa_q8_decode_shared — one decode step of a batch whose sequences all begin
 * with the same prefix, cached once.
 *
 * Sequence s attends over the prefix rows 0 .. prefix_len[0]-1, then over its
 * own rows 0 .. lens[s]-1.  The prefix is read for the whole batch, many
 * sequences' queries per pass over a tile; the two parts of each output are
 * joined by their log-sum-exps, which is exact.  (mqa_decode_beam shares a
 * prefix between the beams of one sequence, over a bf16 cache.)
 *
 *   o, q              device [b, h, d]  (bf16)
 *   prefix_k/v codes  device [m_p, g, d], exponents [g, m_p]
 *   prefix_len        device int32 [1]  (clamped to [0, m_p])
 *   k/v codes         device [b, m_s, g, d], exponents [b, g, m_s]
 *   lens              device int32 [b]  (clamped to [0, m_s])
 *   workspace         device, mqa_q8_decode_shared_workspace_size(b, h, g,
 *                     m_p, d) bytes, as for mqa_q8_decode; among it the prefix
 *                     in fp16, unpacked anew by every call
 *
 * MQA_FLAG_LEN_CLAMPED reports lengths outside [0, m]; 0 is a length here.
 * The prefix's keys and values are exact down to 2^-15 of the largest key or
 * value scale among the 64 rows from a multiple of 64 on; rows of smaller scales
 * are off by up to 2^-25 of it.  Their weights are off by at most 2^-11 of
 * themselves or 2^-27 of the largest p_t s_t, s_t that largest scale; such scales
 * of one K/V head are at most 2^126 apart, and 64 rows of zeros count as 2^-60 of
 * the first that is none of zeros.  The own rows are taken as by mqa_q8_decode.
 * A sequence with no rows at all gets a zero row.  Built for bf16, d = 128
 * and h/g <= 64 (MQA_ERR_UNSUPPORTED otherwise).
 */
MQA_API size_t mqa_q8_decode_shared_workspace_size(int b, int h, int g, int m_p, int d);
MQA_API mqa_status_t mqa_q8_decode_shared(void* o, const void* q, const void* prefix_k, const uint8_t* prefix_k_exps,
                                          const void* prefix_v, const uint8_t* prefix_v_exps,
                                          const int32_t* prefix_len, const void* k_codes, const uint8_t* k_exps,
                                          const void* v_codes, const uint8_t* v_exps, const int32_t* lens, int b,
                                          int h, int g, int m_p, int m_s, int d, float scale, mqa_dtype_t dtype,
                                          void* workspace, size_t workspace_bytes, int32_t* status_flags,
                                          cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMQA_MQA_Q8_H */

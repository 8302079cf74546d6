/*
 * lora_rotary.h -- C ABI of rotary positions (GB300, sm_103a): queries and keys of a decoder layer
 * rotated by their tokens' positions, between the q/k projections and the cache (lora_kv.h, whose
 * lora_kv_write_rotary does it on the way into the cache).
 *
 * A head's first R = rotary_dim values are R / 2 pairs; pair i of a token at position p is turned by
 * the angle a = p freq[i] and multiplied by `factor`:
 *     (x, y)  ->  factor (x cos a - y sin a,  x sin a + y cos a)
 * Values R.. of the head stay as they are. Pair i is values (i, i + R / 2) (LORA_ROTARY_HALF) or
 * (2 i, 2 i + 1) (LORA_ROTARY_INTERLEAVED).
 *
 * The angle is reduced in fixed point: freq[i] / 2 pi is held as a fraction of 2^64 turns, so p times it
 * modulo one turn is exact, and a far position costs no precision: an angle is off by less than 2^-22
 * (plus 2^-51 |p freq[i]|, the roundings of freq[i] and of its quotient in fp64). Sine, cosine and the
 * products are fp32, and a result is rounded once.
 */
#ifndef LORA_ROTARY_H
#define LORA_ROTARY_H

#include "lora_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_ROTARY_MAX_DIM 256   /* largest rotary_dim and head_dim               */
#define LORA_ROTARY_MAX_TENSORS 4 /* tensors of one lora_rotary call               */

typedef enum { LORA_ROTARY_HALF = 0, LORA_ROTARY_INTERLEAVED = 1 } lora_rotary_layout;

/* What lora_rotary_frequencies does to freq[i] = base^(-2 i / R), to use a model at `scale` times
 * the context of `trained` tokens it was trained for. turns_i = trained freq[i] / 2 pi. */
typedef enum {
    LORA_ROTARY_PLAIN = 0,  /* nothing                                                          */
    LORA_ROTARY_LINEAR = 1, /* freq / scale                                                     */
    LORA_ROTARY_NTK = 2,    /* base scale^(R / (R - 2)) in place of base (R > 2)                */
    LORA_ROTARY_YARN = 3,   /* freq for pairs of more than options[0] (32) turns, freq / scale for those
                               of fewer than options[1] (1), linear in i between; the ends are whole
                               i, rounded outwards; factor = 0.1 ln(scale) + 1 (scale > 1)        */
    LORA_ROTARY_BANDS = 4   /* freq / scale below options[0] (1) turns, freq above options[1] (4),
                               linear in turns between                                          */
} lora_rotary_scaling;

/* A rotation: plain host memory, filled by lora_rotary_init and read by the calls when they are
 * made (a captured graph keeps what it was captured with). Nothing to release. */
typedef struct lora_rotary {
    int32_t rotary_dim, layout;
    float factor;
    int32_t reserved;
    uint64_t step[LORA_ROTARY_MAX_DIM / 2]; /* freq[i] / 2 pi, modulo 1, times 2^64          */
} lora_rotary;

/* One tensor of a call: bf16 [T][heads][head_dim], the heads of a token contiguous, `stride` elements from
 * one token to the next (a multiple of 8, at least heads * head_dim), pointers 16-byte aligned. out == in
 * (with the same stride) rotates in place; otherwise the two do not overlap. */
typedef struct lora_rotary_tensor {
    const void *in;
    void *out;
    int64_t in_stride, out_stride;
    int32_t heads, reserved;
} lora_rotary_tensor;

/* HOST: the frequencies of a model. freq: HOST double[rotary_dim / 2]; options: HOST double[2], or NULL
 * for the values in brackets above; scale and trained are read where the scaling says so. *factor
 * receives the factor. Needs no GPU. Errors: ARG (null pointers, an unknown scaling, base or scale or trained not
 * positive and finite, options[0] not above options[1] (YARN) or not below it (BANDS)), SHAPE. */
lora_status lora_rotary_frequencies(int rotary_dim, double base, int scaling, double scale, double trained,
                                    const double *options, double *freq, double *factor);

/* HOST: a rotation by freq (HOST double[rotary_dim / 2], angles from one position to the next).
 * rotary_dim: a multiple of 16, at most LORA_ROTARY_MAX_DIM. Needs no GPU. Errors: ARG (null pointers, an unknown
 * layout, a value that is not finite), SHAPE (rotary_dim). */
lora_status lora_rotary_init(int rotary_dim, int layout, const double *freq, double factor, lora_rotary *out);

/*
 * Rotate n tensors (HOST array, 1..LORA_ROTARY_MAX_TENSORS) of T tokens whose positions are positions[T] (device
 * int32; any values, negative ones turn back), on the current device. head_dim: a multiple of 16, at least
 * rotary_dim, at most LORA_ROTARY_MAX_DIM. inverse != 0: by -a, with the same factor: the inverse for factor
 * 1, and always the gradient (of what comes out with respect to what went in).
 * Asynchronous on `stream`. Errors: ARG, SHAPE (head_dim), UNSUPPORTED, CUDA.
 */
lora_status lora_rotary_apply(const lora_rotary *rotary, int n, const lora_rotary_tensor *tensors, int head_dim,
                              const int32_t *positions, int T, int inverse, lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ROTARY_H */

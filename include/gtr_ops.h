/*
 * gtr_ops.h -- types shared by the operators around the token mixer (gtr_ssm.h,
 * gtr_norm.h), in the same library as gtr_gla.h (libgtr_gla.so).
 */
#ifndef GTR_OPS_H
#define GTR_OPS_H

#include "gtr_gla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of the activations of a call (16 bits each). */
typedef enum { GTR_F16 = 0, GTR_BF16 = 1 } gtr_dtype_t;

/* Activation applied to a result; silu(t) = t / (1 + exp(-t)). */
typedef enum { GTR_ACT_NONE = 0, GTR_ACT_SILU = 1 } gtr_act_t;

#ifdef __cplusplus
}
#endif

#endif /* GTR_OPS_H */

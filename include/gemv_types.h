/*
 * gemv_types.h -- the element types that the entry points for several tokens
 * (include/gemv_tokens.h) and for the key-value cache
 * (include/gemv_attention.h) take by value, next to the types that the entry
 * points of include/gemv.h have in their names.
 */
#ifndef MBGR_GEMV_TYPES_H
#define MBGR_GEMV_TYPES_H

typedef enum gemv_dtype {
    GEMV_F32 = 0,  /* IEEE 754 binary32                                  */
    GEMV_F16 = 1,  /* IEEE 754 binary16                                  */
    GEMV_BF16 = 2  /* bfloat16: the upper 16 bits of a binary32          */
} gemv_dtype;

#endif /* MBGR_GEMV_TYPES_H */

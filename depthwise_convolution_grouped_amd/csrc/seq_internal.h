// Internal interface between the host side of the sequence operators
// (seq_host.cpp) and their kernels.  The public ABI is include/gconv.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include <hip/hip_runtime.h>

#include "gconv.h"

namespace gconv {

// hipLaunchKernel with the arguments converted to the kernel's own parameter
// types; returns this launch's own status.
template <class T> struct same { using type = T; };
template <typename... KP>
hipError_t start(void (*k)(KP...), unsigned grid, unsigned block, unsigned lds, hipStream_t s,
                 typename same<KP>::type... args)
{
    void *argv[] = {(void *)&args...};
    return hipLaunchKernel((const void *)k, dim3(grid), dim3(block), argv, lds, s);
}

// Workgroups of `block` threads in one launch: a runtime refuses 2^32 work-items or more.
constexpr long long most_blocks(unsigned block) { return 0xffffffffll / block; }

inline bool on(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline long long up(long long a, long long b) { return (a + b - 1) / b; }

// v, an fp32 number, in T.  A multiply-add right before a conversion to fp16 may
// become one instruction, which rounds the exact sum to fp16 without a stop at
// fp32; whether it does goes by what else is in the block, so the bits of a
// result would depend on the kernel.  Behind the barrier it is always two.
template <typename T> __device__ __forceinline__ T rounded(float v)
{
    if constexpr (std::is_same<T, _Float16>::value) asm("" : "+v"(v));
    return (T)v;
}

namespace glr {
struct Fwd {
    const void *x, *r, *i;
    const float *lambda, *h0;
    const int32_t *lengths;
    void *y;
    float *h_last, *states, *ws;
};
struct Bwd {
    const void *x, *r, *i;
    const float *lambda;
    const int32_t *lengths;
    const float *states;
    const void *dy;
    const float *dh_last;
    void *dx, *dr, *di;
    float *dlambda, *dh0, *ws;
};
// A validated descriptor.  Workspace sizes in bytes.
size_t fwd_workspace(const gconv_glr_desc &d);
size_t bwd_workspace(const gconv_glr_desc &d);
size_t bwd_min_workspace(const gconv_glr_desc &d);
bool fits(const gconv_glr_desc &d, bool backward);
hipError_t fwd(const gconv_glr_desc &d, const Fwd &a, size_t ws_bytes, hipStream_t s);
hipError_t bwd(const gconv_glr_desc &d, const Bwd &a, size_t ws_bytes, hipStream_t s);
}  // namespace glr

namespace rowq8 {
// x, residual and sum are of d.dtype; weight null: rows as they are.
hipError_t run(const gconv_q8_desc &d, const void *x, const void *residual, const float *weight, int8_t *q,
               float *scale, void *sum, hipStream_t s);
}

namespace mmq8 {
size_t workspace(const gconv_mm_q8_desc &d);
const char *kernel(const gconv_mm_q8_desc &d, const void *a, const void *w, const void *ws, size_t ws_bytes);
hipError_t run(const gconv_mm_q8_desc &d, const int8_t *a, const float *a_scale, const int8_t *w,
               const float *w_scale, const float *bias, void *y, void *ws, size_t ws_bytes, hipStream_t s);
}

}  // namespace gconv

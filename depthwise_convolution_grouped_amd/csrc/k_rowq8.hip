// Rows of 8-bit integers with a scale each, after an optional residual
// addition and root-mean-square norm:
//
//   s = round(x + residual),  v = s rsqrt(mean s^2 + eps) weight,  scale = max |v| / 127,  q = rint(v / scale)
//
// The norm's factor is one number for the row, so max |v| is that factor
// times max |s weight| and cancels from q = rint(s weight * 127 / max |s
// weight|): one reduction over the row (sum of squares and maximum together)
// instead of two, and the row stays in registers between its load and its
// stores.  Memory is all that counts: 8192 x 4096 bf16 with a residual 42 us, 5.6
// TB/s, the rate of a large copy; one row 2.8 us.
#include "device_common.h"
#include "seq_internal.h"

namespace gconv {
namespace rowq8 {
namespace {

constexpr float kLeast = 7.52316385e-37f;   // 2^-120: 127 / kLeast is still finite
// A mean of squares (and eps) below kFaint may have lost bits to fp32's range:
// 2^-126, a square's loss, is 2^-26 of it.  Such a row is summed again times kUp:
// its sum, below 2^-69 for any D, stays finite times kUp^2, and the square of
// fp32's least value, 2^-298, is 2^-110 then.
constexpr float kFaint = 7.88860905e-31f;   // 2^-100
constexpr float kUp = 1.98070406e28f;       // 2^94

template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

struct Params {
    const void *x, *res;
    const float *weight;
    int8_t *q;
    float *scale;
    void *sum;
    long long sx, sr, ss, sq;
    int D;
    float eps, inv_d;
};

// The magnitude's bits compare as integers, and NaN's are the largest.
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }

// The block's sum and maximum, in every thread.
template <int NT> __device__ __forceinline__ void reduce(float &sq, unsigned &top)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        sq += __shfl_xor(sq, o);
        top = umax(top, (unsigned)__shfl_xor((int)top, o));
    }
    if (NT == 64) return;
    constexpr int NW = NT / 64;
    __shared__ float ls[NW];
    __shared__ unsigned lt[NW];
    if (threadIdx.x % 64 == 0) ls[threadIdx.x / 64] = sq, lt[threadIdx.x / 64] = top;
    __syncthreads();
    sq = ls[0];
    top = lt[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) sq += ls[w], top = umax(top, lt[w]);
}

// Whether the sum of squares has to be taken again, the same in every thread.
__device__ __forceinline__ bool faint(const Params &p, float sq, unsigned top)
{
    return sq * p.inv_d + p.eps < kFaint && top < 0x7f800000u && __uint_as_float(top) >= kLeast;
}

// The row's scale and the factor from s * weight to q.  up: sq is that of s * kUp.
template <bool NORM> __device__ __forceinline__ void factors(const Params &p, float sq, unsigned top, bool up, float &scale, float &k)
{
    const float big = __uint_as_float(top);
    const bool bad = top >= 0x7f800000u || (NORM && !(sq < __builtin_inff()));
    if (NORM && up) {   // big, the factor and kUp may pass fp32's range by pairs
        const float norm = 1.0f / sqrtf(sq * p.inv_d + p.eps * kUp * kUp);
        scale = (float)((double)big * (double)norm * ((double)kUp / 127.0));
    } else {
        const float norm = NORM ? 1.0f / sqrtf(sq * p.inv_d + p.eps) : 1.0f;
        scale = big * norm * (1.0f / 127.0f);
    }
    scale = bad ? __builtin_nanf("") : big < kLeast ? 0.0f : scale;
    k = bad || big < kLeast ? 0.0f : 127.0f / big;
}
// q of one value: a NaN or Inf of a row without a scale gives 0.
__device__ __forceinline__ int code(float v, float k) { return k == 0.0f ? 0 : (int)rintf(v * k); }

// Eight channels from ch on, as one piece where the row has eight more; zeros
// past its end.  ALIGNED: D, the strides and the addresses are multiples of
// eight elements.  A channel belongs to the same thread either way, so the
// strides do not change a result's bits.
template <bool ALIGNED, typename T> __device__ __forceinline__ Pack<T, 8> load8(const T *row, int ch, int D)
{
    Pack<T, 8> v;
    if (ALIGNED) {
        v = *(const Pack<T, 8> *)(row + ch);
    } else if (ch + 8 <= D) {
        __builtin_memcpy(&v, row + ch, sizeof(v));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.v[j] = ch + j < D ? row[ch + j] : (T)0.0f;
    }
    return v;
}
template <bool ALIGNED, typename T> __device__ __forceinline__ void store8(T *row, int ch, int D, const Pack<T, 8> &v)
{
    if (ALIGNED) {
        *(Pack<T, 8> *)(row + ch) = v;
    } else if (ch + 8 <= D) {
        __builtin_memcpy(row + ch, &v, sizeof(v));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (ch + j < D) row[ch + j] = v.v[j];
    }
}

// s of one channel once more, after the thread has stored its sums (which may lie over x or the residual).
template <typename T> __device__ __forceinline__ float stored_sum(const T *x, const T *res, const T *sum, long long ch)
{
    if (sum) return to_f32(sum[ch]);
    return res ? to_f32(from_f32<T>(to_f32(x[ch]) + to_f32(res[ch]))) : to_f32(x[ch]);
}

// A row in registers: NT threads with NV pieces of eight channels each.
template <typename T, int NT, int NV, bool NORM, bool ALIGNED> __global__ __launch_bounds__(NT) void held_k(Params p)
{
    using Pk = Pack<T, 8>;
    const long long m = blockIdx.x;
    const T *x = (const T *)p.x + m * p.sx;
    const T *res = p.res ? (const T *)p.res + m * p.sr : nullptr;
    T *sum = p.sum ? (T *)p.sum + m * p.ss : nullptr;
    float s[NV][8];
    float sq = 0.0f;
    unsigned top = 0;
    Pk xv[NV], rv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int ch = (j * NT + (int)threadIdx.x) * 8;
        if (ch < p.D) {
            xv[j] = load8<ALIGNED>(x, ch, p.D);
            if (NORM && res) rv[j] = load8<ALIGNED>(res, ch, p.D);
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int ch = (j * NT + (int)threadIdx.x) * 8;
        if (ch >= p.D) continue;
        Pack<float, 8> w;
        if (NORM) w = load8<ALIGNED>(p.weight, ch, p.D);
        if (NORM && res) {
#pragma unroll
            for (int v = 0; v < 8; ++v) xv[j].v[v] = from_f32<T>(to_f32(xv[j].v[v]) + to_f32(rv[j].v[v]));
            if (sum) store8<ALIGNED>(sum, ch, p.D, xv[j]);
        }
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            float t = to_f32(xv[j].v[v]);
            if (NORM) {
                sq = fmaf(t, t, sq);
                t *= w.v[v];
            }
            s[j][v] = t;
            top = umax(top, mag(t));
        }
    }
    reduce<NT>(sq, top);
    const bool up = NORM && faint(p, sq, top);
    if (up) {
        sq = 0.0f;
#pragma unroll 1
        for (int j = 0; j < NV; ++j) {
            const int c0 = (j * NT + (int)threadIdx.x) * 8;
#pragma unroll 1
            for (int ch = c0; ch < c0 + 8 && ch < p.D; ++ch) {
                const float t = stored_sum(x, res, sum, ch) * kUp;
                sq = fmaf(t, t, sq);
            }
        }
        __syncthreads();   // the first sums have been read
        unsigned none = 0;
        reduce<NT>(sq, none);
    }
    float scale, k;
    factors<NORM>(p, sq, top, up, scale, k);
    if (threadIdx.x == 0) p.scale[m] = scale;
    int8_t *q = p.q + m * p.sq;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int ch = (j * NT + (int)threadIdx.x) * 8;
        if (ch >= p.D) continue;
        Pack<int8_t, 8> o;
#pragma unroll
        for (int v = 0; v < 8; ++v) o.v[v] = (int8_t)code(s[j][v], k);
        store8<ALIGNED>(q, ch, p.D, o);
    }
}

// A row of any length, read twice.  The second reading takes x and the
// residual again unless the sum was stored over one of them; it then reads
// the sum.
template <typename T, bool NORM> __global__ __launch_bounds__(1024) void long_k(Params p)
{
    const long long m = blockIdx.x;
    const T *x = (const T *)p.x + m * p.sx;
    const T *res = p.res ? (const T *)p.res + m * p.sr : nullptr;
    T *sum = p.sum ? (T *)p.sum + m * p.ss : nullptr;
    float sq = 0.0f;
    unsigned top = 0;
    for (long long ch = threadIdx.x; ch < p.D; ch += 1024) {
        T t = x[ch];
        if (NORM && res) t = from_f32<T>(to_f32(t) + to_f32(res[ch]));
        if (NORM && sum) sum[ch] = t;
        float f = to_f32(t);
        if (NORM) {
            sq = fmaf(f, f, sq);
            f *= p.weight[ch];
        }
        top = umax(top, mag(f));
    }
    reduce<1024>(sq, top);
    const bool up = NORM && faint(p, sq, top);
    if (up) {
        sq = 0.0f;
        for (long long ch = threadIdx.x; ch < p.D; ch += 1024) {
            const float t = stored_sum(x, res, sum, ch) * kUp;
            sq = fmaf(t, t, sq);
        }
        __syncthreads();   // the first sums have been read
        unsigned none = 0;
        reduce<1024>(sq, none);
    }
    float scale, k;
    factors<NORM>(p, sq, top, up, scale, k);
    if (threadIdx.x == 0) p.scale[m] = scale;
    for (long long ch = threadIdx.x; ch < p.D; ch += 1024) {   // each thread reads what it wrote itself
        float f = NORM ? stored_sum(x, res, sum, ch) * p.weight[ch] : to_f32(x[ch]);
        p.q[m * p.sq + ch] = (int8_t)code(f, k);
    }
}

// A block a row, in as many launches as their work-items' limit asks for.
template <typename T> hipError_t rows(void (*k)(Params), unsigned block, Params p, long long M, hipStream_t s)
{
    const long long most = most_blocks(block);
    for (;; M -= most) {
        const hipError_t e = start(k, (unsigned)(M < most ? M : most), block, 0, s, p);
        if (e != hipSuccess || M <= most) return e;
        p.x = (const T *)p.x + most * p.sx;
        if (p.res) p.res = (const T *)p.res + most * p.sr;
        if (p.sum) p.sum = (T *)p.sum + most * p.ss;
        p.q += most * p.sq;
        p.scale += most;
    }
}

template <typename T, bool NORM, bool ALIGNED> hipError_t launch(const Params &p, long long M, hipStream_t s)
{
    if (p.D <= 512) return rows<T>(held_k<T, 64, 1, NORM, ALIGNED>, 64, p, M, s);
    if (p.D <= 2048) return rows<T>(held_k<T, 256, 1, NORM, ALIGNED>, 256, p, M, s);
    if (p.D <= 4096) return rows<T>(held_k<T, 256, 2, NORM, ALIGNED>, 256, p, M, s);
    if (p.D <= 8192) return rows<T>(held_k<T, 256, 4, NORM, ALIGNED>, 256, p, M, s);
    if (p.D <= 16384) return rows<T>(held_k<T, 512, 4, NORM, ALIGNED>, 512, p, M, s);
    return rows<T>(long_k<T, NORM>, 1024, p, M, s);
}

template <typename T> hipError_t launch(const Params &p, long long M, bool aligned, hipStream_t s)
{
    if (p.weight) return aligned ? launch<T, true, true>(p, M, s) : launch<T, true, false>(p, M, s);
    return aligned ? launch<T, false, true>(p, M, s) : launch<T, false, false>(p, M, s);
}

}  // namespace

hipError_t run(const gconv_q8_desc &d, const void *x, const void *residual, const float *weight, int8_t *q,
               float *scale, void *sum, hipStream_t s)
{
    Params p{x, residual, weight, q, scale, sum, d.x_stride, residual ? d.residual_stride : 0, sum ? d.sum_stride : 0,
             d.q_stride, (int)d.D, d.eps, 1.0f / (float)d.D};
    const bool aligned = (p.D | p.sx | p.sr | p.ss | p.sq) % 8 == 0 && on(x, 16) && on(residual, 16) &&
                         on(sum, 16) && on(weight, 16) && on(q, 8);
    switch (d.dtype) {
    case GCONV_F32: return launch<float>(p, d.M, aligned, s);
    case GCONV_F16: return launch<_Float16>(p, d.M, aligned, s);
    default: return launch<__bf16>(p, d.M, aligned, s);
    }
}

}  // namespace rowq8
}  // namespace gconv

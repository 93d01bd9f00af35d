// Gated linear recurrence over time, forward and backward:
//
//   log a_t = -c softplus(lambda) sigmoid(r_t),   u_t = sigmoid(i_t) x_t,   m_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + m_t u_t
//
// Steps compose: running steps s .. t takes h_{s-1} to A h_{s-1} + H, and two
// runs join as (A2 A1, A2 H1 + H2).  A block covers 64 channels, one a lane;
// each of its waves reduces a run of S steps to (A, H) in registers, the block
// exchanges the pairs through LDS, and every wave composes those before its
// own and walks its run again, still from registers, with the right state.
// One pass over the data.
//
// The gradient g_t of h_t is the same recurrence from the end: with R_t =
// a_t g_t, g_t = dy_t + R_{t+1}; a run takes R to P R + Q with P = A.  The
// backward pass starts from the states that the forward pass kept every
// GCONV_GLR_SPAN steps and recomputes the rest: no gate or state of a single
// step is ever in memory.  With the state h before the step,
//
//   w_t = R_t log a_t (h_{t-1} - a_t u_t / m_t)      dr = (1 - sigmoid(r)) w
//   dx = g m sigmoid(i)      di = g m u (1 - sigmoid(i))      dlambda = sigmoid(lambda) / softplus(lambda) sum w
//
// and w = 0 where log a = 0 (the limit of log a / sqrt(1 - a^2) at a = 1).
//
// Where rows and channels alone do not fill the chip, the time axis is split
// into chunks.  Forward, in the same launch: a block publishes its (A, H),
// takes those of the chunks before it as they appear, and composes them in
// their order, so the result's bits do not depend on who came first.  A pair
// is one 64-bit word that no pair can equal until it is written: it needs no
// flag and no fence.  The blocks of one row and its channels take their chunks
// from a counter of their own, so a block waits only for blocks that have
// begun, and those publish before they wait themselves.  (One counter for all
// is a queue: 1 x 16384 x 2048 80 us instead of 72, 1 x 4096 x 1024 18 instead
// of 13.)  Backward, where P and Q come from r and dy alone, a kernel of its
// own reduces every chunk first: its pairs handed on as in the forward pass,
// 64 steps a block, 1 x 16384 x 2048 takes 182 us instead of 147.
#include <type_traits>

#include "device_common.h"
#include "seq_internal.h"

// Products and sums join only where it is written: what the compiler makes of
// them goes by basic blocks, and a result's bits would depend on the strides.
#pragma clang fp contract(off)

namespace gconv {
namespace glr {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kLog2eLow = (float)(1.44269504088896340736 - (double)kLog2e);
constexpr int kLanes = 64;    // channels of a block
constexpr int kRuns = 8;      // waves of a block, each with a run of steps
constexpr int kFwdRun = 16, kBwdRun = 8;
constexpr int kFwdStep = kRuns * kFwdRun, kBwdStep = kRuns * kBwdRun;
static_assert(kFwdStep % GCONV_GLR_SPAN == 0 && GCONV_GLR_SPAN % kFwdRun == 0 && kBwdStep % GCONV_GLR_SPAN == 0,
              "kept states lie at the beginnings of runs, and a backward block begins at one");

struct Params {
    const void *x, *r, *i, *dy;
    void *y, *dx, *dr, *di;
    const float *lambda, *h0;   // h0: dh_last in the backward pass
    const int32_t *lengths;
    float *h_last, *states;     // h_last: dh0 in the backward pass
    unsigned *ticket;           // [B][tiles][kApart]: blocks begun (time axis split)
    unsigned long long *pairs;  // [B][nchunk][D], in the order of their use
    unsigned long long *heads;  // [B][ceil(nchunk / kGroup)][D]
    float *part;                // [B][nchunk][D], sums of w
    long long sx[2], sr[2], si[2], sy[2], sdx[2], sdr[2], sdi[2];
    int B, L, D, nspan;
    int clen, nchunk, tiles;    // steps of a chunk, chunks, blocks along the channels
    float c;
};

// log(1 + e^v) = max(v, 0) + log(1 + e) with e = e^-|v|, the logarithm as 2
// atanh(q), q = e / (2 + e) <= 1/3: its series to q^15, below 2e-9 relative.
// (The library's expf and log1pf take 100 instructions, as many as four steps
// of the recurrence.)  t's rounding error, |v| 2^-24, enters as a factor.
__device__ __forceinline__ float softplus(float v)
{
    const float n = fabsf(v) > 150.0f ? -150.0f : -fabsf(v);
    const float t = n * kLog2e, lost = fmaf(n, kLog2eLow, fmaf(n, kLog2e, -t));
    float e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e, lost * kLn2, e);
    const float q = e * __builtin_amdgcn_rcpf(2.0f + e), z = q * q;
    float s = 2.0f / 15;
    s = fmaf(s, z, 2.0f / 13);
    s = fmaf(s, z, 2.0f / 11);
    s = fmaf(s, z, 2.0f / 9);
    s = fmaf(s, z, 2.0f / 7);
    s = fmaf(s, z, 2.0f / 5);
    s = fmaf(s, z, 2.0f / 3);
    s = fmaf(s, z, 2.0f);
    return fmaf(q, s, fmaxf(v, 0.0f));
}

// What a step does, from its gate inputs; `rate` is -c softplus(lambda) log2 e,
// so that y = log2 a.  1 - a^2 is -expm1(2 ln 2 y): its series where y > -0.09
// (2 log a > -0.125: below 5e-8 relative), the difference itself below, where
// it loses about three bits.
struct Gate {
    float e, s, y, a, w;
};
__device__ __forceinline__ Gate decay(float r, float rate)
{
    Gate g;
    g.e = __builtin_amdgcn_exp2f(-kLog2e * r);
    g.s = __builtin_amdgcn_rcpf(1.0f + g.e);
    g.y = rate * g.s;
    g.a = __builtin_amdgcn_exp2f(g.y);
    return g;
}
// The same with an a below 2^-126 as it is, where the instruction makes it 0: log a
// times it may be a gradient above (2% of the backward pass's time).
__device__ __forceinline__ Gate decay_whole(float r, float rate)
{
    Gate g = decay(r, rate);
    g.a = exp2f(g.y);
    return g;
}
constexpr float series(int k)   // the coefficient of y^k in -expm1(2 ln 2 y)
{
    float c = -1.0f;
    for (int j = 1; j <= k; ++j) c *= 1.38629436111989061883f / (float)j;
    return c;
}
__device__ __forceinline__ void power(Gate &g)
{
    float p = fmaf(g.y, series(5), series(4));
    p = fmaf(g.y, p, series(3));
    p = fmaf(g.y, p, series(2));
    p = fmaf(g.y, p, series(1));
    g.w = g.y > -0.09f ? g.y * p : fmaf(-g.a, g.a, 1.0f);
}
// Finite unless lambda is NaN, so that a closed gate (sigmoid 0) gives a = 1 for every lambda.
__device__ __forceinline__ float rate_of(float lambda, float c)
{
    const float rate = -c * softplus(lambda) * kLog2e;
    return rate < -3e38f ? -3e38f : rate;
}

template <typename P> __device__ __forceinline__ int row_length(const P &p, int b)
{
    if (!p.lengths) return p.L;
    const int n = p.lengths[b];
    return n < 0 ? 0 : n > p.L ? p.L : n;
}

// A loaded value stays as its bits, one register each, until it is needed:
// arrays of 16-bit types are packed into pairs as soon as they arrive, which
// waits for them.
template <typename T> __device__ __forceinline__ unsigned bits(T v)
{
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(unsigned, v);
    } else {
        return __builtin_bit_cast(unsigned short, v);
    }
}
template <typename T> __device__ __forceinline__ float value(unsigned b)
{
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(float, b);
    } else {
        return to_f32(__builtin_bit_cast(T, (unsigned short)b));
    }
}
// One tensor from a block's first step on.  `base` and every step's offset are
// the same in all lanes: a load is one instruction with the base in a buffer
// descriptor, the offset in a scalar register and the channel in a vector one,
// where 64-bit addresses cost two or three vector instructions each.  A lane
// that is to store nothing has its channel past the descriptor's end, so that
// stores need no branch: behind one, a wait for the loads before them would
// have to be one for the stores as well.  ONCE: what is loaded is not wanted
// again; such loads, and all stores, go past the caches' older lines (3% of the
// time at 256 MB; the loads that two kernels share stay).  FAR: offsets may pass 31 bits, and
// addresses are computed.
constexpr unsigned kEnd = 0x80000000u;
constexpr int kStream = 2;   // the instruction's bit for that
template <typename T, bool FAR, bool ONCE = true> struct Steps {
    char *base;
    unsigned ch;
    long long step;
    bool live;
    __device__ __forceinline__ Steps(const void *t, const long long *stride, int b, int t0, int ch0, bool stores = true)
        : base((char *)t + (b * stride[0] + t0 * stride[1]) * (long long)sizeof(T)), ch((unsigned)ch0 * sizeof(T)),
          step(stride[1] * (long long)sizeof(T)), live(stores)
    {
        if (!FAR && !stores) ch = kEnd;
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc() const
    {
        return __builtin_amdgcn_make_buffer_rsrc(base, 0, (int)kEnd, 0x00020000);
    }
    // the bits of the value k steps after the first
    __device__ __forceinline__ unsigned load(int k) const
    {
        if constexpr (FAR) {
            T v = *(const T *)(base + k * step + ch);
            return bits(v);
        } else if constexpr (sizeof(T) == 4) {
            return __builtin_amdgcn_raw_buffer_load_b32(rsrc(), ch, (unsigned)k * (unsigned)step, ONCE ? kStream : 0);
        } else {
            return __builtin_amdgcn_raw_buffer_load_b16(rsrc(), ch, (unsigned)k * (unsigned)step, ONCE ? kStream : 0);
        }
    }
    __device__ __forceinline__ void store(int k, T v) const
    {
        if constexpr (FAR) {
            if (live) *(T *)(base + k * step + ch) = v;
        } else if constexpr (sizeof(T) == 4) {
            __builtin_amdgcn_raw_buffer_store_b32(bits(v), rsrc(), ch, (unsigned)k * (unsigned)step, kStream);
        } else {
            __builtin_amdgcn_raw_buffer_store_b16((unsigned short)bits(v), rsrc(), ch, (unsigned)k * (unsigned)step, kStream);
        }
    }
};

// The same number, which the compiler takes for a new one: a run's offsets are
// then added up where they are used and not all kept from before the loop, in
// more scalar registers than there are.
__device__ __forceinline__ int here(int k)
{
    asm volatile("" : "+s"(k));
    return k;
}

// Loads do not move behind this to where their values are used: all of a run's are on their way together.
__device__ __forceinline__ void loads_begin() { asm volatile("" ::: "memory"); }

// ------------------------------------------------- chunks of the time axis

constexpr unsigned long long kNone = ~0ull;   // a word without a pair yet
constexpr int kApart = 16;                    // counters lie 64 bytes apart

__device__ __forceinline__ int up_d(int a, int b) { return (a + b - 1) / b; }

__global__ __launch_bounds__(256) void clear_k(unsigned *ticket, int chains, unsigned long long *pairs, long long n)
{
    const long long k = (long long)blockIdx.x * 256 + threadIdx.x;
    if (k < chains) ticket[k * kApart] = 0;
    if (k < n) pairs[k] = kNone;
}

__device__ __forceinline__ void publish(unsigned long long *to, float a, float h)
{
    unsigned ua = __float_as_uint(a);
    if (ua == 0xffffffffu) ua = 0x7fc00000u;   // any NaN but the one that kNone holds
    const unsigned long long w = (unsigned long long)ua << 32 | __float_as_uint(h);
    __hip_atomic_store(to, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The pair at `from` once it is there.  The wait is bounded (about a second, where
// it is microseconds in use) and ends in NaN.
__device__ __forceinline__ float2 await(const unsigned long long *from)
{
    unsigned long long w = kNone;
    for (int k = 0; k < (1 << 20); ++k) {
        w = __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (w != kNone) break;
        __builtin_amdgcn_s_sleep(1);
    }
    return make_float2(__uint_as_float((unsigned)(w >> 32)), __uint_as_float((unsigned)w));
}

// The state that the chunk `order` in order of use starts from.  The first
// chunk's pair holds the state before it as well, and the last chunk of every
// kGroup publishes its end state, so that no more than kGroup words are read;
// each wave takes a run of them and they join through a and q.
constexpr int kGroup = 16;

typedef float Shared[kRuns][kLanes];   // one value of every wave and lane

// A state through a run (a, h).  The product of a run's decays may be below
// fp32's range where none of them is: 0 times an infinite state would be NaN,
// where step by step the state stays infinite.
__device__ __forceinline__ float through(float a, float s, float h)
{
    return fabsf(s) == __builtin_inff() ? s + h : fmaf(a, s, h);
}

// (A, H) of every wave, joined in the waves' order and applied to `state`;
// mine: the state before this wave's.  Where any lane's comes out NaN, all are
// taken through the runs with more care: 8 x 2048 x 2048 backward takes 109 us
// so, 113 with a branch for each lane and 115 with care always.
template <bool BACK> __device__ __forceinline__ float join_runs(const Shared &a, const Shared &h, int lane, int wave, float &state)
{
    const float from = state;
    float mine = from;
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
        const int j = BACK ? kRuns - 1 - k : k;
        if (j == wave) mine = state;
        state = fmaf(a[j][lane], state, h[j][lane]);
    }
    if (__builtin_amdgcn_ballot_w64(state != state)) {
        state = mine = from;
#pragma unroll 1
        for (int k = 0; k < kRuns; ++k) {
            const int j = BACK ? kRuns - 1 - k : k;
            if (j == wave) mine = state;
            state = through(a[j][lane], state, h[j][lane]);
        }
    }
    return mine;
}
__device__ __forceinline__ float join(const Shared &a, const Shared &h, int lane, int wave, float &state)
{
    return join_runs<false>(a, h, lane, wave, state);
}
// The same from the last wave to the first: the backward pass.
__device__ __forceinline__ float join_back(const Shared &a, const Shared &q, int lane, int wave, float &state)
{
    return join_runs<true>(a, q, lane, wave, state);
}

__device__ __forceinline__ float gather(const Params &p, int b, int ch, int order, int lane, int wave, Shared &a, Shared &q)
{
    const int group = order / kGroup * kGroup;
    const bool head = group > 0;
    const int count = order - group + head;   // words, the head's before the pairs'
    const unsigned long long *pair = p.pairs + ((long long)b * p.nchunk + group - head) * p.D + ch;
    const unsigned long long *heads = p.heads + ((long long)b * up_d(p.nchunk, kGroup) + group / kGroup - 1) * p.D + ch;
    const int per = (count + kRuns - 1) / kRuns;
    const int lo = wave * per, hi = lo + per < count ? lo + per : count;
    float A = 1.0f, H = 0.0f;
    for (int k = lo; k < hi; ++k) {
        const float2 w = await(head && k == 0 ? heads : pair + (long long)k * p.D);
        H = through(w.x, H, w.y);
        A *= w.x;
    }
    a[wave][lane] = A;
    q[wave][lane] = H;
    __syncthreads();
    float state = 0.0f;
    join(a, q, lane, wave, state);
    return state;
}

// ------------------------------------------------------------- forward

// 268 MB in and out take 64 us (1 x 16384 x 2048, split; 4.2 TB/s), of which the
// same loads and stores alone, in 128-byte rows, take 54; the vector units are
// busy 67% of the time.
// SPLIT: a block takes one chunk of kFwdStep steps; else it walks its row's
// whole time in such strides.  (Loads of a stride begun during the one before
// gain nothing: 8 x 2048 x 2048 takes 75 us either way.)
template <typename T, bool SPLIT, bool FAR> __global__ __launch_bounds__(kLanes *kRuns, 4) void fwd_k(Params p)
{
    using In = Steps<T, FAR>;
    constexpr int S = kFwdRun, STEP = kFwdStep;
    __shared__ Shared lds_a[2], lds_h[2];
    __shared__ unsigned lds_id;
    const int lane = threadIdx.x % kLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const unsigned chains = p.tiles * p.B, chain = SPLIT ? blockIdx.x % chains : blockIdx.x;
    const int tile = chain % (unsigned)p.tiles, b = chain / (unsigned)p.tiles;
    const int ch0 = tile * kLanes + lane;
    const bool live = ch0 < p.D;
    const int ch = live ? ch0 : p.D - 1;   // lanes past D repeat its last channel and store nothing
    // the chunk is the block's number among those of its chain, in order of
    // beginning; what does not go by it is loaded while it is on its way
    unsigned number = 0;
    if (SPLIT && threadIdx.x == 0)
        number = __hip_atomic_fetch_add(p.ticket + chain * kApart, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int n = row_length(p, b);
    const float rate = rate_of(p.lambda[ch], p.c);
    if (SPLIT) {
        if (threadIdx.x == 0) lds_id = number;
        __syncthreads();
    }
    const int chunk = SPLIT ? __builtin_amdgcn_readfirstlane((int)lds_id) : 0;
    const int cs = chunk * STEP, ce = SPLIT && cs + STEP < p.L ? cs + STEP : p.L;
    const long long row = (long long)b * p.D + ch;
    float h = p.h0 && chunk == 0 ? p.h0[row] : 0.0f;
    int buf = 0;
    auto keep = [&](int ts, float v) {
        if (p.states && live && ts < ce && ts % GCONV_GLR_SPAN == 0)
            p.states[((long long)b * p.nspan + ts / GCONV_GLR_SPAN) * p.D + ch] = v;
    };
    // FULL: all of the block's steps lie before the row's end
    auto stride = [&](int t0, auto whole) {
        constexpr bool FULL = decltype(whole)::value;
        const int w0 = here(wave * S), ts = t0 + w0;
        const In x(p.x, p.sx, b, t0, ch), r(p.r, p.sr, b, t0, ch), i(p.i, p.si, b, t0, ch), y(p.y, p.sy, b, t0, ch, live);
        unsigned xv[S], rv[S], iv[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {   // steps past the row's end read its last one
            const int k = FULL || ts + s < n ? w0 + s : n - 1 - t0;
            rv[s] = r.load(k), iv[s] = i.load(k), xv[s] = x.load(k);
        }
        loads_begin();
        float a[S], u[S], v[S], A = 1.0f, H = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool in = FULL || ts + s < n;
            a[s] = in ? value<T>(rv[s]) : -__builtin_inff();   // with r = -inf and zeros, a = 1 and nothing enters
            u[s] = in ? value<T>(iv[s]) : 0.0f;
            v[s] = in ? value<T>(xv[s]) : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            Gate g = decay(a[s], rate);
            power(g);
            const float si = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * u[s]));
            a[s] = g.a;
            u[s] = __builtin_amdgcn_sqrtf(g.w) * si * v[s];
            H = fmaf(a[s], H, u[s]);
            A *= a[s];
        }
        lds_a[buf][wave][lane] = A;
        lds_h[buf][wave][lane] = H;
        __syncthreads();
        const bool onward = SPLIT && t0 + STEP < n && wave == 0 && live;   // a chunk of this row follows
        if (onward) {
            float at = chunk == 0 ? 0.0f : 1.0f, ht = h;
#pragma unroll
            for (int j = 0; j < kRuns; ++j) {
                const float ja = lds_a[buf][j][lane];
                ht = through(ja, ht, lds_h[buf][j][lane]);
                at *= ja;
            }
            publish(p.pairs + ((long long)b * p.nchunk + chunk) * p.D + ch, at, ht);
        }
        if (SPLIT && chunk > 0) h = gather(p, b, ch, chunk, lane, wave, lds_a[1], lds_h[1]);
        float hs = join(lds_a[buf], lds_h[buf], lane, wave, h);
        if (onward && chunk % kGroup == kGroup - 1)
            publish(p.heads + ((long long)b * up_d(p.nchunk, kGroup) + chunk / kGroup) * p.D + ch, 0.0f, h);
        keep(ts, hs);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            hs = fmaf(a[s], hs, u[s]);
            if (FULL || ts + s < ce) y.store(w0 + s, rounded<T>(FULL || ts + s < n ? hs : 0.0f));
        }
        buf ^= 1;
    };
    int t0 = cs;
    for (; t0 < ce && t0 + STEP <= n; t0 += STEP) stride(t0, std::true_type());
    if (t0 < ce && t0 < n) stride(t0, std::false_type()), t0 += STEP;
    for (; t0 < ce; t0 += STEP) {   // past the row's end, for the whole block
        const int w0 = wave * S, ts = t0 + w0;
        const In y(p.y, p.sy, b, t0, ch, live);
        for (int s = 0; s < S; ++s)
            if (ts + s < ce) y.store(w0 + s, rounded<T>(0.0f));
        keep(ts, 0.0f);
    }
    // the block that holds the row's end has its last state
    if (p.h_last && wave == 0 && live && (!SPLIT || chunk == (n > 0 ? (n - 1) / STEP : 0))) p.h_last[row] = h;
}

// What a few steps need: 328 bytes of arguments cost the host 0.8 us more than
// 96.  The other kernels keep Params: with smaller arguments of its own the
// compiler gives fwd_k 84 registers instead of 70, and a compute unit holds two
// blocks instead of three (1 x 16384 x 2048 68 -> 75 us).
struct Few {
    const void *x, *r, *i;
    void *y;
    const float *lambda, *h0;
    const int32_t *lengths;
    float *h_last, *states;
    long long sx[2], sr[2], si[2], sy[2];
    int L, D, nspan, tiles;
    float c;
};

// A few steps: one thread takes its channel through all of them.  One step of 1 x
// 2048 channels takes 3 us, of 128 x 4096 5 us: a launch and one trip to memory.
template <typename T> __global__ __launch_bounds__(64) void fwd_serial_k(Few p)
{
    const unsigned bid = blockIdx.x;
    const int tile = bid % (unsigned)p.tiles, b = bid / (unsigned)p.tiles;
    const int ch = tile * 64 + (int)threadIdx.x;
    if (ch >= p.D) return;
    const T *x = (const T *)p.x + b * p.sx[0] + ch;
    const T *r = (const T *)p.r + b * p.sr[0] + ch;
    const T *i = (const T *)p.i + b * p.si[0] + ch;
    T *y = (T *)p.y + b * p.sy[0] + ch;
    const int n = row_length(p, b);
    const long long row = (long long)b * p.D + ch;
    float h = p.h0 ? p.h0[row] : 0.0f;
    const float rate = rate_of(p.lambda[ch], p.c);
    for (int t = 0; t < p.L; ++t) {
        if (p.states && t % GCONV_GLR_SPAN == 0) p.states[((long long)b * p.nspan + t / GCONV_GLR_SPAN) * p.D + ch] = h;
        if (t < n) {
            Gate g = decay(to_f32(r[t * p.sr[1]]), rate);
            power(g);
            const float si = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * to_f32(i[t * p.si[1]])));
            h = fmaf(g.a, h, __builtin_amdgcn_sqrtf(g.w) * si * to_f32(x[t * p.sx[1]]));
        }
        y[t * p.sy[1]] = rounded<T>(t < n ? h : 0.0f);
    }
    if (p.h_last) p.h_last[row] = h;
}

// ------------------------------------------------------------ backward

// What a chunk makes of R: pairs[b][chunk] = (P, Q).  The chunk with the row's
// end takes dh_last in (P = 0).  The first chunk's is not wanted: its place
// takes dh_last to the last chunk's block of the next kernel, whose first
// chunk's block may write dh0 over it.
template <typename T, bool FAR> __global__ __launch_bounds__(kLanes *kRuns) void bwd_reduce_k(Params p)
{
    using In = Steps<T, FAR, false>;
    constexpr int S = kBwdRun, STEP = kBwdStep;
    __shared__ Shared lds_a[2], lds_q[2];
    const int lane = threadIdx.x % kLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const int tile = blockIdx.x % (unsigned)p.tiles, rest = blockIdx.x / (unsigned)p.tiles;
    const int chunk = rest % (p.nchunk - 1) + 1, b = rest / (p.nchunk - 1);
    const int ch0 = tile * kLanes + lane;
    const bool live = ch0 < p.D;
    const int ch = live ? ch0 : p.D - 1;
    const int n = row_length(p, b), cs = chunk * p.clen, end = cs + p.clen < n ? cs + p.clen : n;
    if (cs >= n) return;
    const bool tail = n <= cs + p.clen;
    const float rate = rate_of(p.lambda[ch], p.c);
    float R = tail && p.h0 ? p.h0[(long long)b * p.D + ch] : 0.0f, at = tail ? 0.0f : 1.0f;
    if (tail && wave == 0 && live) p.pairs[(long long)b * p.nchunk * p.D + ch] = __float_as_uint(R);
    int buf = 0;
    auto stride = [&](int t0, auto whole) {
        constexpr bool FULL = decltype(whole)::value;
        const int w0 = here(wave * S), ts = t0 + w0, most = n - 1 - t0;
        const In r(p.r, p.sr, b, t0, ch), dy(p.dy, p.sy, b, t0, ch);
        unsigned rv[S], gv[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int k = FULL || w0 + s < most ? w0 + s : most;
            rv[s] = r.load(k), gv[s] = dy.load(k);
        }
        loads_begin();
        float A = 1.0f, Q = 0.0f;
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
            if (!FULL && ts + s >= n) continue;
            const float a = decay(value<T>(rv[s]), rate).a;
            Q = a * (value<T>(gv[s]) + Q);
            A *= a;
        }
        lds_a[buf][wave][lane] = A;
        lds_q[buf][wave][lane] = Q;
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int j = kRuns - 1; j >= 0; --j) {
                const float ja = lds_a[buf][j][lane];
                R = through(ja, R, lds_q[buf][j][lane]);
                at *= ja;
            }
        }
        buf ^= 1;
    };
    int t0 = cs + (end - cs - 1) / STEP * STEP;
    if (t0 + STEP > n) stride(t0, std::false_type()), t0 -= STEP;
    for (; t0 >= cs; t0 -= STEP) stride(t0, std::true_type());
    if (wave == 0 && live)
        p.pairs[((long long)b * p.nchunk + chunk) * p.D + ch] =
            (unsigned long long)__float_as_uint(at) << 32 | __float_as_uint(R);
}

// 8 x 2048 x 2048 takes 113 us, 4.2 TB/s of seven tensors, the vector units busy
// 65% of the time.
// A block takes one chunk, the whole row where there is one.  AHEAD: it begins
// a stride's loads while it works on the one before, in half as many registers
// again: 134 -> 117 us for 8 x 2048 x 2048 (one block a compute unit), 101 ->
// 116 us for 12 x 1024 x 2048 (more).
template <typename T, bool FAR, bool AHEAD> __global__ __launch_bounds__(kLanes *kRuns, AHEAD ? 2 : 4) void bwd_k(Params p)
{
    using In = Steps<T, FAR>;
    constexpr int S = kBwdRun, STEP = kBwdStep;
    __shared__ Shared lds_a[2], lds_h[2], lds_q[2];
    const int lane = threadIdx.x % kLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    const int tile = blockIdx.x % (unsigned)p.tiles, rest = blockIdx.x / (unsigned)p.tiles;
    const int chunk = rest % p.nchunk, b = rest / p.nchunk;
    const int ch0 = tile * kLanes + lane;
    const bool live = ch0 < p.D;
    const int ch = live ? ch0 : p.D - 1;
    const int n = row_length(p, b);
    const int cs = chunk * p.clen, ce = cs + p.clen < p.L ? cs + p.clen : p.L;
    const int tail = n > 0 ? (n - 1) / p.clen : 0;   // the chunk with the row's end
    const long long row = (long long)b * p.D + ch;
    const float rate = rate_of(p.lambda[ch], p.c);
    float R = 0.0f, sum = 0.0f;
    if (chunk == tail) {
        if (tail > 0) R = __uint_as_float((unsigned)p.pairs[(long long)b * p.nchunk * p.D + ch]);
        else if (p.h0) R = p.h0[row];
    }
    if (chunk < tail) {   // what the chunks after this one make of it: each wave composes a run of their pairs
        const int count = tail - chunk, per = (count + kRuns - 1) / kRuns;
        const int lo = wave * per, hi = lo + per < count ? lo + per : count;
        const unsigned long long *pair = p.pairs + ((long long)b * p.nchunk + chunk + 1) * p.D + ch;
        float A = 1.0f, Q = 0.0f;
        for (int k = hi - 1; k >= lo; --k) {
            const unsigned long long w = pair[(long long)k * p.D];
            const float a = __uint_as_float((unsigned)(w >> 32));
            Q = through(a, Q, __uint_as_float((unsigned)w));
            A *= a;
        }
        lds_a[1][wave][lane] = A;
        lds_q[1][wave][lane] = Q;
        __syncthreads();
        join_back(lds_a[1], lds_q[1], lane, wave, R);
    }
    unsigned xv[S], rv[S], iv[S], gv[S];
    float hn = 0.0f;
    auto load = [&](int t0, auto whole) {   // steps past the row's end read its last one
        constexpr bool FULL = decltype(whole)::value;
        const In x(p.x, p.sx, b, t0, ch), r(p.r, p.sr, b, t0, ch), i(p.i, p.si, b, t0, ch), dy(p.dy, p.sy, b, t0, ch);
        const int w0 = here(wave * S), most = n - 1 - t0;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int k = FULL || w0 + s < most ? w0 + s : most;
            rv[s] = r.load(k), iv[s] = i.load(k), xv[s] = x.load(k), gv[s] = dy.load(k);
        }
        hn = p.states[((long long)b * p.nspan + t0 / GCONV_GLR_SPAN) * p.D + ch];
        loads_begin();
    };
    int buf = 0, t0 = cs + (ce - cs - 1) / STEP * STEP;
    for (; t0 >= cs && t0 >= n; t0 -= STEP) {   // past the row's end, for the whole block
        const In dx(p.dx, p.sdx, b, t0, ch, live), dr(p.dr, p.sdr, b, t0, ch, live), di(p.di, p.sdi, b, t0, ch, live);
        for (int k = wave * S; k < wave * S + S; ++k)
            if (t0 + k < ce) {
                dx.store(k, rounded<T>(0.0f));
                dr.store(k, rounded<T>(0.0f));
                di.store(k, rounded<T>(0.0f));
            }
    }
    if (AHEAD && t0 >= cs) load(t0, std::false_type());
    // FULL: all of the block's steps lie before the row's end
    auto stride = [&](int t0, auto whole) {
        constexpr bool FULL = decltype(whole)::value;
        const int w0 = here(wave * S), ts = t0 + w0;
        const In dx(p.dx, p.sdx, b, t0, ch, live), dr(p.dr, p.sdr, b, t0, ch, live), di(p.di, p.sdi, b, t0, ch, live);
        if (!AHEAD) load(t0, whole);
        // of every step: a, log2 a, m sigmoid(i), both 1 - sigmoid, m u, and a u / m
        float a[S], la[S], ms[S], nr[S], ni[S], bu[S], d[S], gy[S], A = 1.0f, H = 0.0f, Q = 0.0f, hs = hn;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool in = FULL || ts + s < n;
            a[s] = in ? value<T>(rv[s]) : -__builtin_inff();   // with r = -inf and zeros, R and h pass
            ni[s] = in ? value<T>(iv[s]) : 0.0f;
            bu[s] = in ? value<T>(xv[s]) : 0.0f;
            gy[s] = in ? value<T>(gv[s]) : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            Gate k = decay_whole(a[s], rate);
            power(k);
            const float ei = __builtin_amdgcn_exp2f(-kLog2e * ni[s]);
            const float si = __builtin_amdgcn_rcpf(1.0f + ei);
            // at w = 0 (log a = 0, or so small that w is no normal number) m is 0, and so is log a / m
            const float im = k.w > 1e-37f ? __builtin_amdgcn_rsqf(k.w) : 0.0f;
            const float u = si * bu[s], m = k.w * im;
            a[s] = k.a;
            la[s] = k.y;
            ms[s] = m * si;
            bu[s] = m * u;
            d[s] = u * im * k.a;
            nr[s] = fminf(k.e * k.s, 1.0f);   // 1 for infinity times 0; a gate's NaN comes through la and bu
            ni[s] = fminf(ei * si, 1.0f);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            H = fmaf(a[s], H, bu[s]);
            A *= a[s];
            Q = a[S - 1 - s] * (gy[S - 1 - s] + Q);
        }
        lds_a[buf][wave][lane] = A;
        lds_h[buf][wave][lane] = H;
        lds_q[buf][wave][lane] = Q;
        if (AHEAD && t0 - STEP >= cs) load(t0 - STEP, std::true_type());
        __syncthreads();
        for (int j = 0; j < wave; ++j) hs = fmaf(lds_a[buf][j][lane], hs, lds_h[buf][j][lane]);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            d[s] = hs - d[s];
            hs = fmaf(a[s], hs, bu[s]);
            ni[s] *= bu[s];
        }
        float Rs = join_back(lds_a[buf], lds_q[buf], lane, wave, R);
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
            const bool in = FULL || ts + s < n;
            const float g = gy[s] + Rs;
            Rs = a[s] * g;
            const float w = in ? Rs * la[s] * d[s] : 0.0f, gin = in ? g : 0.0f;
            sum += w;
            if (FULL || ts + s < ce) {
                dx.store(w0 + s, rounded<T>(gin * ms[s]));
                dr.store(w0 + s, rounded<T>(nr[s] * (w * kLn2)));
                di.store(w0 + s, rounded<T>(gin * ni[s]));
            }
        }
        buf ^= 1;
    };
    if (t0 >= cs && t0 + STEP > n) stride(t0, std::false_type()), t0 -= STEP;
    for (; t0 >= cs; t0 -= STEP) stride(t0, std::true_type());
    __syncthreads();
    lds_q[0][wave][lane] = sum * kLn2;
    __syncthreads();
    if (wave == 0 && live) {
        float t = 0.0f;
        for (int j = 0; j < kRuns; ++j) t += lds_q[0][j][lane];
        p.part[((long long)b * p.nchunk + chunk) * p.D + ch] = t;
        if (chunk == 0 && p.h_last) p.h_last[row] = R;
    }
}

// dlambda of n channels from the blocks' sums of w, rows of D, added in order: 32 threads a channel
// take every 32nd row each, then one joins them.  4.6 us for 16 rows of 2048, a
// launch's time; the last block of bwd_k to end doing it instead gains nothing
// (1 x 16384 x 2048 147 us either way).
__global__ __launch_bounds__(1024) void dlambda_k(const float *part, const float *lambda, float *dlambda, long long rows,
                                                  int D, int n)
{
    __shared__ float lds[32][33];
    const int lane = threadIdx.x % 32, sub = threadIdx.x / 32, ch = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (ch < n) {
#pragma unroll 4
        for (long long k = sub; k < rows; k += 32) t += part[k * D + ch];
    }
    lds[sub][lane] = t;
    __syncthreads();
    if (sub || ch >= n) return;
    t = 0.0f;
    for (int j = 0; j < 32; ++j) t += lds[j][lane];
    const float l = lambda[ch], sp = softplus(l), e = expf(-fabsf(l));
    const float sig = (l >= 0.0f ? 1.0f : e) / (1.0f + e);
    dlambda[ch] = (sp > 0.0f ? sig / sp : 1.0f) * t;
}

// No step at all (L = 0): the state, or its gradient, passes through.
__global__ __launch_bounds__(256) void pass_k(const float *from, float *to, long long n)
{
    const long long k = (long long)blockIdx.x * 256 + threadIdx.x;
    if (k < n) to[k] = from ? from[k] : 0.0f;
}

// ---------------------------------------------------------------- host

constexpr int kSerial = 8;              // steps that one thread takes alone

// The time axis is split where there are few blocks without it.  Forward, below
// 512 and from three chunks on (8 x 2048 x 2048, 256 blocks: 67 us, 74 whole; 16
// x 1024 x 2048, 512 blocks: 64 and 60; 1 x 200 x 4096, two chunks: 12 and 10).
// Backward, below 256, into chunks that make kBwdBlocks (8 x 2048 x 2048: 120
// us, 117 whole; 1 x 16384 x 2048: 147 us with 512 or 1024 blocks, 183 with
// 256).  kAhead: the blocks that run at once, one a compute unit.
constexpr long long kFwdSplit = 512, kBwdSplit = 256, kBwdBlocks = 512;
constexpr unsigned kAhead = 256;

struct Shape {
    int tiles, clen, nchunk;
};

Shape whole(const gconv_glr_desc &d) { return {(int)up(d.D, kLanes), (int)d.L, 1}; }

Shape fwd_shape(const gconv_glr_desc &d)
{
    Shape s = whole(d);
    if (d.L > 2 * kFwdStep && s.tiles * d.B < kFwdSplit) s.clen = kFwdStep, s.nchunk = (int)up(d.L, kFwdStep);
    return s;
}

Shape bwd_shape(const gconv_glr_desc &d)
{
    Shape s = whole(d);
    const long long blocks = s.tiles * d.B;
    if (d.L > kBwdStep && blocks > 0 && blocks < kBwdSplit) {
        const long long strides = up(d.L, kBwdStep), chunks = up(kBwdBlocks, blocks);
        s.clen = (int)(up(strides, chunks < strides ? chunks : strides) * kBwdStep);
        s.nchunk = (int)up(d.L, s.clen);
    }
    return s;
}

size_t words(const gconv_glr_desc &d, const Shape &s) { return (size_t)d.B * (s.nchunk + up(s.nchunk, kGroup)) * d.D; }
size_t tickets(const gconv_glr_desc &d, const Shape &s) { return (size_t)s.tiles * d.B * kApart * sizeof(unsigned); }
size_t fwd_bytes(const gconv_glr_desc &d, const Shape &s)   // the tickets, the pairs and the heads
{
    return s.nchunk > 1 ? tickets(d, s) + words(d, s) * sizeof(unsigned long long) : 0;
}
size_t bwd_pairs(const gconv_glr_desc &d, const Shape &s)
{
    return s.nchunk > 1 ? (size_t)d.B * s.nchunk * d.D * sizeof(unsigned long long) : 0;
}
size_t bwd_parts(const gconv_glr_desc &d, const Shape &s) { return (size_t)d.B * s.nchunk * d.D * sizeof(float); }

Params params(const gconv_glr_desc &d, const Shape &s)
{
    Params p{};
    for (int k = 0; k < 2; ++k) {
        p.sx[k] = d.x_stride[k];
        p.sr[k] = d.r_stride[k];
        p.si[k] = d.i_stride[k];
        p.sy[k] = d.y_stride[k];
        p.sdx[k] = d.dx_stride[k];
        p.sdr[k] = d.dr_stride[k];
        p.sdi[k] = d.di_stride[k];
    }
    p.B = (int)d.B;
    p.L = (int)d.L;
    p.D = (int)d.D;
    p.c = d.c;
    p.nspan = (int)up(d.L, GCONV_GLR_SPAN);
    p.clen = s.clen;
    p.nchunk = s.nchunk;
    p.tiles = s.tiles;
    return p;
}

// A launch's grid times its block stays below 2^32, so what may need more goes
// in ranges: batch rows (whole rows, n of them from b on), and of split rows the
// blocks, which take their chunks' numbers from counters and go on where the
// launch before stopped.
Params rows_from(Params p, long long b, long long n, long long e)
{
    auto move = [&](auto &t, const long long *stride) {
        if (t) t = (std::remove_reference_t<decltype(t)>)((char *)t + b * stride[0] * e);
    };
    move(p.x, p.sx), move(p.r, p.sr), move(p.i, p.si), move(p.y, p.sy), move(p.dy, p.sy);
    move(p.dx, p.sdx), move(p.dr, p.sdr), move(p.di, p.sdi);
    if (p.lengths) p.lengths += b;
    if (p.h0) p.h0 += b * p.D;
    if (p.h_last) p.h_last += b * p.D;
    if (p.states) p.states += b * p.nspan * p.D;
    if (p.part) p.part += b * p.D;
    p.B = (int)n;
    return p;
}

// f(Params of a range, its grid) for all batch rows, the time axis whole.
template <typename F> hipError_t whole_rows(const gconv_glr_desc &d, const Params &p, unsigned block, long long e, F &&f)
{
    const long long most = most_blocks(block) / p.tiles;
    if (d.B <= most) return f(p, (unsigned)(p.tiles * d.B));
    for (long long b = 0; b < d.B; b += most) {
        const long long n = d.B - b < most ? d.B - b : most;
        const hipError_t r = f(rows_from(p, b, n, e), (unsigned)(p.tiles * n));
        if (r != hipSuccess) return r;
    }
    return hipSuccess;
}

template <typename T, bool FAR> hipError_t fwd_t(const gconv_glr_desc &d, const Shape &sh, Params p, void *ws, hipStream_t st)
{
    constexpr unsigned block = kLanes * kRuns;
    if (d.L <= kSerial)
        return whole_rows(d, p, 64, sizeof(T), [&](const Params &q, unsigned grid) {
            const Few f{q.x, q.r, q.i, q.y, q.lambda, q.h0, q.lengths, q.h_last, q.states,
                        {q.sx[0], q.sx[1]}, {q.sr[0], q.sr[1]}, {q.si[0], q.si[1]}, {q.sy[0], q.sy[1]},
                        q.L, q.D, q.nspan, q.tiles, q.c};
            return start(fwd_serial_k<T>, grid, 64, 0, st, f);
        });
    if (p.nchunk == 1)
        return whole_rows(d, p, block, sizeof(T),
                          [&](const Params &q, unsigned grid) { return start(fwd_k<T, false, FAR>, grid, block, 0, st, q); });
    const long long words_all = (long long)words(d, sh), words_most = most_blocks(256) * 256;
    p.ticket = (unsigned *)ws;
    p.pairs = (unsigned long long *)((char *)ws + tickets(d, sh));
    p.heads = p.pairs + (size_t)d.B * sh.nchunk * d.D;
    const long long chains = p.tiles * d.B;
    hipError_t e = hipSuccess;
    for (long long k = 0; k < words_all && e == hipSuccess; k += words_most) {
        const long long n = words_all - k < words_most ? words_all - k : words_most;
        e = start(clear_k, (unsigned)up(n, 256), 256, 0, st, p.ticket, (int)chains, p.pairs + k, n);
    }
    const long long all = chains * p.nchunk, most = most_blocks(block) / chains * chains;
    for (long long k = 0; k < all && e == hipSuccess; k += most)
        e = start(fwd_k<T, true, FAR>, (unsigned)(all - k < most ? all - k : most), block, 0, st, p);
    return e;
}

template <typename T, bool FAR> hipError_t bwd_t(const gconv_glr_desc &d, const Params &p, hipStream_t st)
{
    constexpr unsigned block = kLanes * kRuns;
    if (p.nchunk == 1)
        return whole_rows(d, p, block, sizeof(T), [&](const Params &q, unsigned grid) {
            return p.tiles * d.B <= kAhead ? start(bwd_k<T, FAR, true>, grid, block, 0, st, q)
                                           : start(bwd_k<T, FAR, false>, grid, block, 0, st, q);
        });
    const unsigned row = (unsigned)(p.tiles * d.B);   // below kBwdSplit, with about kBwdBlocks blocks in all
    const hipError_t e = start(bwd_reduce_k<T, FAR>, row * (p.nchunk - 1), block, 0, st, p);
    return e != hipSuccess ? e : start(bwd_k<T, FAR, false>, row * p.nchunk, block, 0, st, p);
}

// No step at all: the state, or its gradient, to where it goes.
hipError_t pass(const float *from, float *to, long long n, hipStream_t s)
{
    const long long most = most_blocks(256) * 256;
    hipError_t e = hipSuccess;
    for (long long k = 0; k < n && e == hipSuccess; k += most) {
        const long long m = n - k < most ? n - k : most;
        e = start(pass_k, (unsigned)up(m, 256), 256, 0, s, from ? from + k : nullptr, to + k, m);
    }
    return e;
}

// f of a value of the element type, and of whether a block's offsets, in
// bytes, need more than 31 bits.
template <typename F> hipError_t by_type(const gconv_glr_desc &d, bool backward, F &&f)
{
    long long most = 0;
    for (long long s : {d.x_stride[1], d.r_stride[1], d.i_stride[1], d.y_stride[1]}) most = s > most ? s : most;
    if (backward)
        for (long long s : {d.dx_stride[1], d.dr_stride[1], d.di_stride[1]}) most = s > most ? s : most;
    const bool far = (most * kFwdStep + d.D) * 4 >= (long long)kEnd;
    auto with = [&](auto t) { return far ? f(t, std::true_type()) : f(t, std::false_type()); };
    return d.dtype == GCONV_F32 ? with(float()) : d.dtype == GCONV_F16 ? with(_Float16()) : with(__bf16());
}

}  // namespace

// One batch row's channels are one launch: blocks of kLanes * kRuns threads hold
// fewer than 2^29 of them, so that a channel's byte offset stays below 2^31.
bool fits(const gconv_glr_desc &d, bool backward)
{
    return (!backward && d.L <= kSerial) || up(d.D, kLanes) <= most_blocks(kLanes * kRuns);
}

size_t fwd_workspace(const gconv_glr_desc &d) { return d.B == 0 || d.L <= kSerial ? 0 : fwd_bytes(d, fwd_shape(d)); }

size_t bwd_workspace(const gconv_glr_desc &d)
{
    if (d.B == 0 || d.L == 0) return 0;
    const Shape s = bwd_shape(d);
    return bwd_pairs(d, s) + bwd_parts(d, s);
}

size_t bwd_min_workspace(const gconv_glr_desc &d) { return d.B == 0 || d.L == 0 ? 0 : bwd_parts(d, whole(d)); }

hipError_t fwd(const gconv_glr_desc &d, const Fwd &a, size_t ws_bytes, hipStream_t s)
{
    if (d.L == 0) {
        if (!a.h_last || a.h_last == a.h0) return hipSuccess;
        return pass(a.h0, a.h_last, d.B * d.D, s);
    }
    Shape sh = fwd_shape(d);
    if (d.L <= kSerial || ws_bytes < fwd_bytes(d, sh) || !on(a.ws, 8)) sh = whole(d);
    Params p = params(d, sh);
    p.x = a.x;
    p.r = a.r;
    p.i = a.i;
    p.y = a.y;
    p.lambda = a.lambda;
    p.h0 = a.h0;
    p.lengths = a.lengths;
    p.h_last = a.h_last;
    p.states = a.states;
    return by_type(d, false, [&](auto t, auto far) { return fwd_t<decltype(t), decltype(far)::value>(d, sh, p, a.ws, s); });
}

hipError_t bwd(const gconv_glr_desc &d, const Bwd &a, size_t ws_bytes, hipStream_t s)
{
    hipError_t e = hipSuccess;
    const float *part = nullptr;
    long long rows = 0;
    if (d.B > 0 && d.L == 0) {
        if (a.dh0 && a.dh0 != a.dh_last) e = pass(a.dh_last, a.dh0, d.B * d.D, s);
    } else if (d.B > 0) {
        Shape sh = bwd_shape(d);
        if (ws_bytes < bwd_pairs(d, sh) + bwd_parts(d, sh) || !on(a.ws, 8)) sh = whole(d);
        Params p = params(d, sh);
        p.x = a.x;
        p.r = a.r;
        p.i = a.i;
        p.dy = a.dy;
        p.dx = a.dx;
        p.dr = a.dr;
        p.di = a.di;
        p.lambda = a.lambda;
        p.h0 = a.dh_last;
        p.lengths = a.lengths;
        p.h_last = a.dh0;
        p.states = const_cast<float *>(a.states);
        p.pairs = (unsigned long long *)a.ws;
        p.part = (float *)((char *)a.ws + bwd_pairs(d, sh));
        part = p.part;
        rows = d.B * sh.nchunk;
        e = by_type(d, true, [&](auto t, auto far) { return bwd_t<decltype(t), decltype(far)::value>(d, p, s); });
    }
    const long long most = most_blocks(1024) * 32;
    for (long long k = 0; k < d.D && e == hipSuccess; k += most) {
        const long long n = d.D - k < most ? d.D - k : most;
        e = start(dlambda_k, (unsigned)up(n, 32), 1024, 0, s, part ? part + k : nullptr, a.lambda + k, a.dlambda + k, rows,
                  (int)d.D, (int)n);
    }
    return e;
}

}  // namespace glr
}  // namespace gconv

// Product of two matrices of 8-bit integers on the matrix cores, both with
// their rows along k and a scale for each row:
//
//   y[m][n] = (sum_k a[m][k] w[n][k]) a_scale[m] w_scale[n] + bias[n]
//
// The sums are 32-bit integers, so no order of summation changes them.  w
// takes the matrix instruction's row side and a its column side: a lane then
// holds runs of four consecutive n of one m, and stores them together.
#include <type_traits>

#include "device_common.h"
#include "seq_internal.h"

namespace gconv {
namespace mmq8 {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Params {
    const int8_t *a, *w;
    const float *sa, *sw, *bias;
    void *y;
    long long la, lw, ly;
    int M, N, K;
    int tm, tn;     // tiles along m and n
};

// One output from its sum.  Every kernel here ends with it, so that a result
// does not depend on the kernel that a call takes.
__device__ __forceinline__ float scaled(int sum, float sa, float sw, float bias)
{
    return fmaf((float)sum * sa, sw, bias);
}

// Up to four outputs of row m from column n on: scaled, rounded once, stored.
template <typename T> __device__ __forceinline__ void store4(const Params &p, int m, int n, i32x4 acc)
{
    if (m >= p.M || n >= p.N) return;
    const float sa = p.sa[m];
    T *y = (T *)p.y + m * p.ly + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= p.N) return;
        y[j] = rounded<T>(scaled(acc[j], sa, p.sw[n + j], p.bias ? p.bias[n + j] : 0.0f));
    }
}

// 16 bytes of a row from k on, zeros from K on; any alignment.
__device__ __forceinline__ i32x4 row16(const int8_t *row, int k, int K)
{
    i32x4 v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else if (k < K) {
        int8_t b[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) b[j] = k + j < K ? row[k + j] : (int8_t)0;
        __builtin_memcpy(&v, b, 16);
    }
    return v;
}

// Any sizes, strides and alignment: 64 x 64 outputs a block, 64 of k a step,
// loaded through registers.
template <typename T> __global__ __launch_bounds__(256) void any_k(Params p)
{
    constexpr int ROW = 80;   // bytes of an LDS row: 64 and a pad that spreads the rows over the banks
    __shared__ __align__(16) int8_t la[64 * ROW], lw[64 * ROW];
    const int tile = blockIdx.x;
    const int m0 = tile % p.tm * 64, n0 = tile / p.tm * 64;
    const int t = threadIdx.x, lane = t % 64, wave = t / 64;
    const int wn = wave % 2 * 32, wm = wave / 2 * 32;
    const int row = t / 4, piece = t % 4 * 16;
    const int ra = m0 + row < p.M ? m0 + row : p.M - 1, rw = n0 + row < p.N ? n0 + row : p.N - 1;
    const int8_t *ap = p.a + ra * p.la, *wp = p.w + rw * p.lw;
    i32x4 acc[2][2] = {};
    i32x4 av = row16(ap, piece, p.K), wv = row16(wp, piece, p.K);
    for (int k0 = 0; k0 < p.K; k0 += 64) {
        __syncthreads();
        *(i32x4 *)(la + row * ROW + piece) = av;
        *(i32x4 *)(lw + row * ROW + piece) = wv;
        __syncthreads();
        if (k0 + 64 < p.K) {
            av = row16(ap, k0 + 64 + piece, p.K);
            wv = row16(wp, k0 + 64 + piece, p.K);
        }
        i32x4 af[2], wf[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            af[j] = *(const i32x4 *)(la + (wm + j * 16 + lane % 16) * ROW + lane / 16 * 16);
            wf[j] = *(const i32x4 *)(lw + (wn + j * 16 + lane % 16) * ROW + lane / 16 * 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[i], af[j], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            store4<T>(p, m0 + wm + j * 16 + lane % 16, n0 + wn + i * 16 + lane / 16 * 4, acc[i][j]);
}

// ---- tiles staged by asynchronous loads
//
// BM x BN outputs a block, 128 bytes of k a step.  LDS is a ring of P panels,
// an operand's rows of one step each, in the order a0 w0 a1 w1 a2 ...: while
// the matrix cores work on two of them, the others are on their way, straight
// from memory to LDS.  A wave owns WM x WN outputs in 32 x 32 x 32
// instructions.
//
// LDS holds rows of 128 bytes as eight pieces of 16; piece c of row r lies at
// place c ^ (r / 2 % 8).  The loads write 64 pieces in lane order (8 rows), so
// a lane fetches the piece that belongs at its place; the reads of one piece
// from 16 consecutive rows then touch each of the 64 banks once.
//
// 8192 x 8192 x 4096 takes 250 us, 2.2 Pop/s, the matrix cores busy 61% of the
// cycles, of which there are 1.8 to the ns; 8192 x 8192 x 8192 2.5 Pop/s.

typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef int rsrc_t __attribute__((ext_vector_type(4)));

constexpr unsigned kOob = 0x80000000u;   // past every descriptor's end: reads zeros

__device__ __forceinline__ rsrc_t make_rsrc(const void *base, unsigned bytes)
{
    const unsigned long long a = (unsigned long long)base;
    rsrc_t r;
    r.x = __builtin_amdgcn_readfirstlane((int)(unsigned)(a & 0xffffffffull));
    r.y = __builtin_amdgcn_readfirstlane((int)(unsigned)((a >> 32) & 0xffffull));
    r.z = __builtin_amdgcn_readfirstlane((int)bytes);
    r.w = 0x00020000;
    return r;
}

// 16 bytes a lane from byte `voffset` + `soffset` to LDS byte lds_byte + 16 * lane.
__device__ __forceinline__ void dma16(unsigned voffset, unsigned soffset, unsigned lds_byte, rsrc_t r)
{
    asm volatile("s_mov_b32 m0, %1\n\t"
                 "s_nop 0\n\t"
                 "buffer_load_dwordx4 %0, %2, %3 offen lds"
                 :
                 : "v"(voffset), "s"(lds_byte), "s"(r), "s"(soffset)
                 : "memory", "m0");
}

// A wave's outputs of 32 rows of m and W columns of n, from LDS (rows of PITCH
// bytes) to memory in whole rows, 16 bytes a lane: parts of a 128-byte line
// written apart cost a third of the rate.  One element at a time where the
// rows are not aligned for that or end inside.
template <typename T, int W, int PITCH>
__device__ __forceinline__ void store_rows(const Params &p, const char *lds, int m, int n, int lane, bool wide)
{
    constexpr int PER = 16 / (int)sizeof(T), PIECES = W / PER, STEP = 64 / PIECES;
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += STEP) {
        const int r = r0 + lane / PIECES, c = lane % PIECES * PER;
        const uint4 v = *(const uint4 *)(lds + r * PITCH + c * sizeof(T));
        if (m + r >= p.M) continue;
        T *y = (T *)p.y + (m + r) * p.ly + n + c;
        if (wide) {
            *(uint4 *)y = v;
        } else {
            T t[PER];
            __builtin_memcpy(t, &v, 16);
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (n + c + j < p.N) y[j] = t[j];
        }
    }
}

template <typename T, int BM, int BN, int WM, int WN, int P>
__global__ __launch_bounds__(BM / WM * (BN / WN) * 64) void tile_k(Params p)
{
    constexpr int NWM = BM / WM, NW = NWM * (BN / WN);
    constexpr int PANEL = (BM > BN ? BM : BN) * 128;
    constexpr int LA = BM / 8 / NW, LW = BN / 8 / NW;     // loads of a wave for one step
    static_assert(LA * NW * 8 == BM && LW * NW * 8 == BN, "");
    constexpr int TM = WM / 32, TN = WN / 32;
    constexpr int PITCH = WN * (int)sizeof(T) + 16, OUT = 32 * PITCH + WN * 8;
    static_assert(NW * OUT <= P * PANEL, "a wave's outputs, scales and biases take the operands' place");
    __shared__ __align__(1024) char lds[P * PANEL];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    // tiles: each XCD takes a run of them, in columns of 8 tiles along m
    const int tile = xcd_tile(blockIdx.x, p.tm * p.tn);
    const int band = tile / (8 * p.tn), first = band * 8;
    const int high = p.tm - first < 8 ? p.tm - first : 8, at = tile - first * p.tn;
    const int m0 = (first + at % high) * BM, n0 = at / high * BN;

    const int rows_a = p.M - m0 < BM ? p.M - m0 : BM, rows_w = p.N - n0 < BN ? p.N - n0 : BN;
    const rsrc_t ra = make_rsrc(p.a + m0 * p.la, (unsigned)((rows_a - 1) * p.la + p.K));
    const rsrc_t rw = make_rsrc(p.w + n0 * p.lw, (unsigned)((rows_w - 1) * p.lw + p.K));
    unsigned oa[LA], ow[LW];
    auto piece = [&](int load) { return (lane % 8 ^ (load % 2 * 4 + lane / 16)) * 16; };
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        const int r = (wave * LA + j) * 8 + lane / 8;
        oa[j] = (unsigned)((r < rows_a ? r : rows_a - 1) * p.la) + piece(wave * LA + j);
    }
#pragma unroll
    for (int j = 0; j < LW; ++j) {
        const int r = (wave * LW + j) * 8 + lane / 8;
        ow[j] = (unsigned)((r < rows_w ? r : rows_w - 1) * p.lw) + piece(wave * LW + j);
    }
    const unsigned base = (unsigned)(size_t)lds;
    // load j of one operand's rows at k into the ring's panel at byte `to`;
    // pieces past K are zeros (the last step's, and all of the steps after it)
    auto load = [&](const unsigned *o, rsrc_t r, int count, int j, int k, int to) {
        unsigned v = o[j];
        if (k + 128 > p.K) v = k + piece(wave * count + j) < p.K ? v : kOob;
        dma16(v, k, base + to + (wave * count + j) * 1024, r);
    };

    const int wm = wave % NWM * WM, wn = wave / NWM * WN;
    const int place = (lane / 32 ^ lane / 2 % 8) * 16;
    const char *fa = lds + (wm + lane % 32) * 128, *fw = lds + (wn + lane % 32) * 128;
    // what the outputs need: WN columns over the lanes, this lane's rows
    const int n = n0 + wn, half = lane / 32;
    const int col = n + lane % WN < p.N ? n + lane % WN : p.N - 1;
    const float sw_col = p.sw[col], bias_col = p.bias ? p.bias[col] : 0.0f;
    float sa[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int m = m0 + wm + j * 32 + lane % 32;
        sa[j] = p.sa[m < p.M ? m : p.M - 1];
    }
    i32x16 acc[TN][TM] = {};
    i32x4 wf[2][TN], af[2][TM];
    auto read = [&](int pa, int pw, int s, int to) {
#pragma unroll
        for (int j = 0; j < TN; ++j) wf[to][j] = *(const i32x4 *)(fw + pw + j * 4096 + (place ^ s * 32));
#pragma unroll
        for (int j = 0; j < TM; ++j) af[to][j] = *(const i32x4 *)(fa + pa + j * 4096 + (place ^ s * 32));
    };
    // A step's reads stay ahead of the products that do not need them, and its
    // loads [l0, l1) go out between products: a burst of them would hold up
    // the waves behind it.
    int k = 0, free = (P - 2) * PANEL;   // the step, and the two panels its loads go to
    auto next = [](int panel) { return panel == (P - 1) * PANEL ? 0 : panel + PANEL; };
    auto multiply = [&](int from, int l0, int l1) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[from][i], af[from][j], acc[i][j], 0, 0, 0);
                const int at = i * TM + j;
#pragma unroll
                for (int l = l0; l < l1; ++l) {
                    if ((l - l0) * (TN * TM) / (l1 - l0) != at) continue;
                    __builtin_amdgcn_sched_barrier(0);
                    const int other = l - (P % 2 ? LW : LA);   // panel P - 2 first, then panel P - 1
                    if (P % 2) {
                        if (other < 0) load(ow, rw, LW, l, k + (P - 3) / 2 * 128, free);
                        else load(oa, ra, LA, other, k + (P - 1) / 2 * 128, next(free));
                    } else {
                        if (other < 0) load(oa, ra, LA, l, k + (P - 2) / 2 * 128, free);
                        else load(ow, rw, LW, other, k + (P - 2) / 2 * 128, next(free));
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        __builtin_amdgcn_sched_barrier(0);
    };
    // the panels that may still be on their way when a step begins: P - 4, a first
    constexpr int LATE = (P - 3) / 2 * LA + (P - 4) / 2 * LW;
#pragma unroll
    for (int c = 0; c < P - 2; ++c) {
#pragma unroll
        for (int j = 0; j < (c % 2 ? LW : LA); ++j) {
            if (c % 2) load(ow, rw, LW, j, c / 2 * 128, c * PANEL);
            else load(oa, ra, LA, j, c / 2 * 128, c * PANEL);
        }
    }
    int pa = 0, pw = PANEL;   // the step's panels
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LATE) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(pa, pw, 0, 0);
    constexpr int LL = LA + LW, L1 = (LL + 2) / 3, L2 = L1 + (LL - L1 + 1) / 2;
    for (;; k += 128) {
        read(pa, pw, 1, 1);
        multiply(0, 0, L1);
        read(pa, pw, 2, 0);
        multiply(1, L1, L2);
        read(pa, pw, 3, 1);
        multiply(0, L2, LL);
        const bool more = k + 128 < p.K;
        if (more) {   // this step is read and the next one has landed, for every wave
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LATE) : "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            free = pa;   // the panels just read
            pa = next(next(pa));
            pw = next(next(pw));
            read(pa, pw, 0, 0);
        }
        multiply(1, 0, 0);
        if (!more) break;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the loads past K have written their zeros
    __syncthreads();

    char *mine = lds + wave * OUT;   // a wave's own
    float *sw = (float *)(mine + 32 * PITCH), *bias = sw + WN;
    sw[lane % WN] = sw_col;
    bias[lane % WN] = bias_col;
    const bool wide = n + WN <= p.N && p.ly % (16 / (int)sizeof(T)) == 0 && ((uintptr_t)p.y & 15) == 0;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
#pragma unroll
        for (int i = 0; i < TN; ++i) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {   // a lane's sums are of four runs of four n, for one m
                const int c = i * 32 + g * 8 + half * 4;
                const float4 w = *(const float4 *)(sw + c), b = *(const float4 *)(bias + c);
                struct alignas(4 * sizeof(T)) { T v[4]; } o;
                o.v[0] = rounded<T>(scaled(acc[i][j][g * 4], sa[j], w.x, b.x));
                o.v[1] = rounded<T>(scaled(acc[i][j][g * 4 + 1], sa[j], w.y, b.y));
                o.v[2] = rounded<T>(scaled(acc[i][j][g * 4 + 2], sa[j], w.z, b.z));
                o.v[3] = rounded<T>(scaled(acc[i][j][g * 4 + 3], sa[j], w.w, b.w));
                __builtin_memcpy(__builtin_assume_aligned(mine + lane % 32 * PITCH + c * sizeof(T), 4 * sizeof(T)), &o, sizeof(o));
            }
        }
        store_rows<T, WN, PITCH>(p, mine, m0 + wm + j * 32, n, lane, wide);
    }
}

// ---- few rows of a
//
// What counts is reading w once, with enough loads in flight.  A block owns
// 16 columns of n and AL * 8 rows of m; its NW waves split k in pieces of 128
// bytes, and the partial sums join in LDS.  A wave's pieces come through a ring
// of its own in LDS, P deep, filled by asynchronous loads of whole 128-byte
// lines: loaded straight into the instruction's layout, 16 bytes of 16 rows
// side by side, a compute unit takes 16 bytes a cycle instead of 64 (48 x 4096
// x 4096 takes 9.6 us that way, 6.9 this way).  The layout of a piece is that
// of the tiles above.  Rows past M and pieces past K are zeros and cost no
// traffic.
template <typename T, int AL, int NW, int P> __global__ __launch_bounds__(NW * 64) void few_k(Params p)
{
    constexpr int MT = (AL + 1) / 2, LOADS = 2 + AL, STAGE = LOADS * 1024, PAD = AL % 2 * 1024, OUT = (MT * 256 + NW * 64 - 1) / (NW * 64);
    static_assert(MT * 1024 <= P * STAGE && (P - 1) * LOADS < 64, "the sums take the ring's place; a count of loads");
    __shared__ __align__(1024) char lds[NW * P * STAGE + PAD];   // a row past the eight of an odd AL is read, for nothing
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int n0 = blockIdx.x % (unsigned)p.tn * 16, m0 = blockIdx.x / (unsigned)p.tn * (MT * 16);
    // what the outputs need: output o of the block is row o / 16, column o % 16
    float sa[OUT], sw[OUT], bias[OUT];
#pragma unroll
    for (int j = 0; j < OUT; ++j) {
        const int o = (int)threadIdx.x + j * NW * 64, m = m0 + o / 16, n = n0 + o % 16;
        const bool in = o < MT * 256 && m < p.M && n < p.N;
        sa[j] = in ? p.sa[m] : 0.0f;
        sw[j] = in ? p.sw[n] : 0.0f;
        bias[j] = in && p.bias ? p.bias[n] : 0.0f;
    }
    const int rows_a = p.M - m0 < AL * 8 ? p.M - m0 : AL * 8, rows_w = p.N - n0 < 16 ? p.N - n0 : 16;
    const rsrc_t ra = make_rsrc(p.a + m0 * p.la, (unsigned)((rows_a - 1) * p.la + p.K));
    const rsrc_t rw = make_rsrc(p.w + n0 * p.lw, (unsigned)((rows_w - 1) * p.lw + p.K));
    // load l of a piece: rows l * 8 to l * 8 + 7 of w, then of a
    unsigned at[LOADS];
#pragma unroll
    for (int l = 0; l < LOADS; ++l) {
        const int r = (l < 2 ? l : l - 2) * 8 + lane / 8, c = (lane % 8 ^ (l % 2 * 4 + lane / 16)) * 16;
        at[l] = r < (l < 2 ? rows_w : rows_a) ? (unsigned)(r * (l < 2 ? p.lw : p.la)) + c : kOob;
    }
    const unsigned base = (unsigned)(size_t)lds + wave * (P * STAGE);
    auto load = [&](int piece) {   // this wave's, by its number
        const int k = (wave + piece * NW) * 128, slot = piece % P * STAGE;
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            unsigned v = at[l];
            if (k + 128 > p.K) v = k + (lane % 8 ^ (l % 2 * 4 + lane / 16)) * 16 < p.K ? v : kOob;
            dma16(v, k, base + slot + l * 1024, l < 2 ? rw : ra);
        }
    };
    const int all = (p.K + 127) / 128, mine = all > wave ? (all - wave + NW - 1) / NW : 0;
    const char *frag = lds + wave * (P * STAGE) + lane % 16 * 128;
    const int place = (lane / 16 ^ lane % 16 / 2) * 16;
    i32x4 acc[MT] = {};
#pragma unroll
    for (int j = 0; j < P - 1; ++j) load(j);
    for (int j = 0; j < mine; ++j) {
        // the slot of the piece before this one has been read
        load(j + P - 1);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((P - 1) * LOADS) : "memory");
        const char *f = frag + j % P * STAGE;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const i32x4 wf = *(const i32x4 *)(f + (place ^ u * 64));
#pragma unroll
            for (int t = 0; t < MT; ++t)
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf, *(const i32x4 *)(f + 2048 + t * 2048 + (place ^ u * 64)), acc[t], 0, 0, 0);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the loads past the last piece have written their zeros
    __syncthreads();
    int *part = (int *)lds;   // [wave][row][column]
#pragma unroll
    for (int t = 0; t < MT; ++t) *(i32x4 *)(part + ((wave * MT + t) * 16 + lane % 16) * 16 + lane / 16 * 4) = acc[t];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < OUT; ++j) {
        const int o = (int)threadIdx.x + j * NW * 64, m = m0 + o / 16, n = n0 + o % 16;
        if (o >= MT * 256 || m >= p.M || n >= p.N) continue;
        int sum = 0;
#pragma unroll
        for (int v = 0; v < NW; ++v) sum += part[v * MT * 256 + o];
        ((T *)p.y)[m * p.ly + n] = rounded<T>(scaled(sum, sa[j], sw[j], bias[j]));
    }
}

// Bytes k to k + 15 of a row of K >= 16, zeros from K on: the 16 that end with the
// row's, shifted, where those would pass its end.  Any alignment.
struct Tail {
    int from, past;   // where to read, and by how many bytes k lies past it
    __device__ __forceinline__ Tail(int k, int K) : from(k < K - 16 ? k : K - 16), past(k - from) {}
    __device__ __forceinline__ i32x4 shifted(i32x4 v) const
    {
        if (past >= 16) return i32x4{0, 0, 0, 0};
        const int words = past / 4;
        int x[5];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = 0;
#pragma unroll
            for (int j = i; j < 4; ++j) x[i] = words == j - i ? v[j] : x[i];
        }
        x[4] = 0;
        i32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (int)__builtin_amdgcn_alignbyte((unsigned)x[i + 1], (unsigned)x[i], (unsigned)past % 4);
        return o;
    }
};

// The same for rows of any stride and alignment, K at least 16: their pieces go
// through registers, a piece ahead of the products, to one place a wave.  16 x
// 4000 x 4095 takes 5.4 us, 333 x 1001 x 1111 6.8.
template <typename T, int MT, int NW> __global__ __launch_bounds__(NW * 64) void few_any_k(Params p)
{
    constexpr int LOADS = (1 + MT) * 2, STAGE = LOADS * 1024, OUT = (MT * 256 + NW * 64 - 1) / (NW * 64);
    static_assert(MT * 1024 <= STAGE, "the sums take the pieces' place");
    __shared__ __align__(1024) char lds[NW * STAGE];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int n0 = blockIdx.x % (unsigned)p.tn * 16, m0 = blockIdx.x / (unsigned)p.tn * (MT * 16);
    float sa[OUT], sw[OUT], bias[OUT];   // output o of the block is row o / 16, column o % 16
#pragma unroll
    for (int j = 0; j < OUT; ++j) {
        const int o = (int)threadIdx.x + j * NW * 64, m = m0 + o / 16, n = n0 + o % 16;
        const bool in = o < MT * 256 && m < p.M && n < p.N;
        sa[j] = in ? p.sa[m] : 0.0f;
        sw[j] = in ? p.sw[n] : 0.0f;
        bias[j] = in && p.bias ? p.bias[n] : 0.0f;
    }
    // load l of a piece: rows l * 8 to l * 8 + 7 of w, then of a; rows past the last repeat it
    const int8_t *row[LOADS];
#pragma unroll
    for (int l = 0; l < LOADS; ++l) {
        const int r = (l < 2 ? n0 + l * 8 : m0 + (l - 2) * 8) + lane / 8, last = (l < 2 ? p.N : p.M) - 1;
        row[l] = (l < 2 ? p.w : p.a) + (r < last ? r : last) * (l < 2 ? p.lw : p.la);
    }
    char *mine = lds + wave * STAGE;
    i32x4 v[LOADS];
    auto load = [&](int k) {   // bytes k to k + 127 of every row, eight lanes a row
        const Tail t(k + lane % 8 * 16, p.K);
#pragma unroll
        for (int l = 0; l < LOADS; ++l) __builtin_memcpy(&v[l], row[l] + t.from, 16);
        if (k + 128 > p.K) {
#pragma unroll
            for (int l = 0; l < LOADS; ++l) v[l] = t.shifted(v[l]);
        }
    };
    const char *frag = mine + lane % 16 * 128;
    const int place = (lane / 16 ^ lane % 16 / 2) * 16;
    i32x4 acc[MT] = {};
    const int first = wave * 128;
    if (first < p.K) load(first);
    for (int k = first; k < p.K; k += NW * 128) {
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const int c = lane % 8 ^ (l % 2 * 4 + lane / 16);   // the layout of the tiles above
            *(i32x4 *)(mine + l * 1024 + lane / 8 * 128 + c * 16) = v[l];
        }
        if (k + NW * 128 < p.K) load(k + NW * 128);
        // the wave's own writes, read by its other lanes: in order, without a barrier of the block
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const i32x4 wf = *(const i32x4 *)(frag + (place ^ u * 64));
#pragma unroll
            for (int t = 0; t < MT; ++t)
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf, *(const i32x4 *)(frag + 2048 + t * 2048 + (place ^ u * 64)), acc[t], 0, 0, 0);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    __syncthreads();
    int *part = (int *)lds;   // [wave][row][column]
#pragma unroll
    for (int t = 0; t < MT; ++t) *(i32x4 *)(part + ((wave * MT + t) * 16 + lane % 16) * 16 + lane / 16 * 4) = acc[t];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < OUT; ++j) {
        const int o = (int)threadIdx.x + j * NW * 64, m = m0 + o / 16, n = n0 + o % 16;
        if (o >= MT * 256 || m >= p.M || n >= p.N) continue;
        int sum = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += part[w * MT * 256 + o];
        ((T *)p.y)[m * p.ly + n] = rounded<T>(scaled(sum, sa[j], sw[j], bias[j]));
    }
}

template <typename T, int AL, int NW, int P> hipError_t few(Params p, hipStream_t s)
{
    p.tm = (int)up(p.M, AL * 8);
    p.tn = (int)up(p.N, 16);
    return start(few_k<T, AL, NW, P>, (unsigned)((long long)p.tm * p.tn), NW * 64, 0, s, p);
}
template <typename T, int MT> hipError_t few_any(Params p, hipStream_t s)
{
    if (p.K < 16) return hipErrorInvalidValue;   // it reads 16 bytes of a row at once
    p.tm = (int)up(p.M, MT * 16);
    p.tn = (int)up(p.N, 16);
    return start(few_any_k<T, MT, 8>, (unsigned)((long long)p.tm * p.tn), 512, 0, s, p);
}

template <typename T, int BM, int BN, int WM, int WN, int P> hipError_t tiles(Params p, hipStream_t s)
{
    p.tm = (int)up(p.M, BM);
    p.tn = (int)up(p.N, BN);
    return start(tile_k<T, BM, BN, WM, WN, P>, (unsigned)((long long)p.tm * p.tn), BM / WM * (BN / WN) * 64, 0, s, p);
}

// ---- rows that are not whole pieces of 16 bytes
//
// Copies rows to rows of `kp` bytes, K rounded up to 16, with zeros past K:
// the tiles then take them as any others.  Both operands in one launch, the
// first `split` pieces a's.
struct Pack {
    const int8_t *from[2];
    long long stride[2], split, pieces;
    int8_t *to;
    int K, per;   // pieces of a row
};
__global__ __launch_bounds__(256) void pack_k(Pack q)
{
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    if (at >= q.pieces) return;
    const int which = at >= q.split;
    const long long mine = which ? at - q.split : at, row = mine / q.per;
    *(i32x4 *)(q.to + at * 16) = row16(q.from[which] + row * q.stride[which], (int)(mine - row * q.per) * 16, q.K);
}

// The time of a tile shape in us, from its measured start and step (128 of k)
// with one block a compute unit and with `side` of them side by side.  Only the
// order of the shapes' times counts: on a full chip the clock goes down, and
// 8192 x 8192 x 4096 takes 250 us where this says 190.
double estimate(const Params &p, int bm, int bn, double start1, double step1, int side, double start2, double step2)
{
    const double n = (double)up(p.M, bm) * up(p.N, bn), steps = (double)up(p.K, 128);
    if (n <= 256 || side == 1) return up((long long)n, 256) * (start1 + step1 * steps);
    return up((long long)n, 256 * side) * (start2 + step2 * steps);
}

// Small tiles fill the chip, large ones read less: 2048 x 2048 x 2048 takes
// 25.1 us with 256 x 256 tiles, 15.2 with 128 x 128 and 19.9 with 64 x 64;
// 8192 x 8192 x 4096 takes 250, 315 and 448; 256 x 4096 x 4096 takes 41.1,
// 22.5 and 12.3.
struct Times {
    double t256, t128, t64;
    explicit Times(const Params &p)
        : t256(estimate(p, 256, 256, 6.0, 1.3, 1, 0, 0)), t128(estimate(p, 128, 128, 4.0, 0.6, 2, 5.0, 1.28)),
          t64(estimate(p, 64, 64, 2.6, 0.27, 2, 3.0, 0.47))
    {
    }
    double least() const { return t64 < t128 ? (t64 < t256 ? t64 : t256) : (t128 < t256 ? t128 : t256); }
};

// The same of few_k with 16 * mt rows a block: a start, what a compute unit's
// blocks take one after the other (their operands come at 100 GB/s, and a
// block after the first has a start of its own, longest where no second one
// fits beside it, at mt = 3), and w from memory.  At N = K = 4096, 16, 32, 48 and
// 64 rows take 5.6, 6.0, 6.9 and 7.9 us, with 64 x 64 tiles 10.5; 128 x 1024 x
// 4096 takes 4.7, with 32 rows a block, and 10.5; 333 x 1024 x 1024 4.7 and 4.9.
double turns(const Params &p, int mt) { return (double)up(up(p.M, mt * 16) * up(p.N, 16), 256); }
double few_time(const Params &p, int mt)
{
    const double n = turns(p, mt), again = mt == 1 ? 0.6 : mt == 2 ? 0.55 : mt == 3 ? 1.8 : 1.2;
    return 1.5 + 0.3 * mt + (n - 1) * again + n * (1 + mt) * 16e-5 * p.K + (double)p.N * p.K / 9e6;
}
int few_best(const Params &p)   // the mt of the least time
{
    int best = 1;
    for (int mt = 2; mt <= 4; ++mt)
        if (few_time(p, mt) < few_time(p, best)) best = mt;
    return best;
}

// What a call runs.  few: up to 8 rows, then 16 * mt a block; tiles: square; lying: rows read as they lie.
enum Kernel { kFew8, kFew16, kFew32, kFew48, kFew64, kTile64, kTile128, kTile256, kLying16, kLying32, kLying64, kAny };

// Rows in whole pieces.  Up to 8 rows a stage of the ring is smaller and there
// are three: 1 x 8192 x 4096 8.5 -> 7.6 us.
Kernel of_pieces(const Params &p)
{
    const Times t(p);
    const int mt = few_best(p);
    if (few_time(p, mt) < t.least()) return p.M <= 8 ? kFew8 : (Kernel)(kFew16 + mt - 1);
    return t.t64 <= t.t128 && t.t64 <= t.t256 ? kTile64 : t.t128 <= t.t256 ? kTile128 : kTile256;
}

// Rows that few_k and tile_k take as they are: whole pieces of 16 bytes, and within a descriptor's reach.
bool fine(const void *a, long long stride, int K) { return K % 16 == 0 && stride % 16 == 0 && on(a, 16) && stride < (1 << 22); }

long long padded(int K) { return up(K, 16) * 16; }

// The time of rows read as they lie, with 64 x 64 tiles (mt = 0: 333 x 1001 x
// 1111 14.7 us, 600 x 4096 x 1001 20.9) or with 16 * mt rows a block (the same 6.8
// with mt = 2, 7.6 with 4, and 24.8 and 22.9), and of copying them first: a copy
// costs about 4 us and a byte of it 1 / 2 MB of a us (10.2 us and 14.5; 200 x 4000 x
// 4095 24, 33 with mt = 4 and 43 with tiles).
constexpr int kLying[] = {1, 2, 4};
double lying_time(const Params &p, int mt)
{
    if (mt == 0) {
        const double blocks = (double)up(p.M, 64) * (double)up(p.N, 64);
        return (0.85 + 0.45 * blocks / 384) * (2.5 + 0.62 * (double)up(p.K, 64));
    }
    const double n = turns(p, mt);
    return mt == 1 ? 2.2 + n * (0.2 + 0.00068 * p.K) : mt == 2 ? 2.4 + n * (0.3 + 0.00102 * p.K) : 3.1 + n * (0.3 + 0.0018 * p.K);
}
int lying_best(const Params &p)
{
    int best = 0;
    if (p.K < 16) return best;   // few_any refuses them
    for (int mt : kLying)
        if (lying_time(p, mt) < lying_time(p, best)) best = mt;
    return best;
}
bool pack_pays(const Params &p)
{
    if (((double)p.M + p.N) * (double)up(p.K, 16) > (double)most_blocks(256) * 256) return false;   // one launch
    const double few = few_time(p, few_best(p)), tiles = Times(p).least();
    return lying_time(p, lying_best(p)) > (few < tiles ? few : tiles) + 4.0 + ((double)p.M + p.N) * p.K / 2e6;
}

struct Route {
    bool a_fine, w_fine, pack;   // pack: the operands that are not fine are copied first
    Kernel kernel;
};
Route route(const Params &p, const void *ws, size_t ws_bytes)
{
    Route r{fine(p.a, p.la, p.K), fine(p.w, p.lw, p.K), false, kAny};
    if (r.a_fine && r.w_fine) {
        r.kernel = of_pieces(p);
        return r;
    }
    const size_t need = ((r.a_fine ? 0 : (size_t)p.M) + (r.w_fine ? 0 : (size_t)p.N)) * padded(p.K);
    r.pack = on(ws, 16) && ws_bytes >= need && pack_pays(p);
    if (r.pack) {
        Params q = p;
        q.K = (int)padded(p.K);
        r.kernel = of_pieces(q);
    } else {
        const int mt = lying_best(p);
        r.kernel = mt == 0 ? kAny : mt == 1 ? kLying16 : mt == 2 ? kLying32 : kLying64;
    }
    return r;
}

template <typename T> hipError_t launch(Params p, void *ws, size_t ws_bytes, hipStream_t s)
{
    const Route r = route(p, ws, ws_bytes);
    if (r.pack) {
        const long long kp = padded(p.K);
        const int per = (int)(kp / 16);
        Pack q{{p.a, p.w}, {p.la, p.lw}, r.a_fine ? 0 : p.M * (long long)per, 0, (int8_t *)ws, p.K, per};
        q.pieces = q.split + (r.w_fine ? 0 : p.N * (long long)per);
        if (!r.a_fine) p.a = q.to, p.la = kp;
        if (!r.w_fine) p.w = q.to + q.split * 16, p.lw = kp;
        const hipError_t e = start(pack_k, (unsigned)up(q.pieces, 256), 256, 0, s, q);
        if (e != hipSuccess) return e;
        p.K = (int)kp;
    }
    switch (r.kernel) {
    case kFew8: return few<T, 1, 8, 3>(p, s);
    case kFew16: return few<T, 2, 8, 2>(p, s);
    case kFew32: return few<T, 4, 4, 2>(p, s);
    case kFew48: return few<T, 6, 8, 2>(p, s);
    case kFew64: return few<T, 8, 4, 2>(p, s);
    case kTile64: return tiles<T, 64, 64, 32, 32, 10>(p, s);
    case kTile128: return tiles<T, 128, 128, 64, 32, 5>(p, s);
    case kTile256: return tiles<T, 256, 256, 128, 64, 5>(p, s);
    case kLying16: return few_any<T, 1>(p, s);
    case kLying32: return few_any<T, 2>(p, s);
    case kLying64: return few_any<T, 4>(p, s);
    case kAny: break;
    }
    p.tm = (int)up(p.M, 64);
    p.tn = (int)up(p.N, 64);
    return start(any_k<T>, (unsigned)((long long)p.tm * p.tn), 256, 0, s, p);
}

// The part of y that a launch may hold (parts() below).
struct Part {
    long long rows, columns;
    explicit Part(const Params &p)
    {
        const long long most = most_blocks(512), m16 = up(p.M, 16), n16 = up(p.N, 16);
        rows = p.M, columns = p.N;
        if (m16 * n16 <= most) return;
        rows = (m16 < 2048 ? m16 : 2048) * 16;
        columns = most / (rows / 16) * 16;
    }
    Params at(const Params &p, long long m, long long n) const
    {
        Params q = p;
        q.M = (int)(p.M - m < rows ? p.M - m : rows);
        q.N = (int)(p.N - n < columns ? p.N - n : columns);
        q.a += m * p.la, q.sa += m, q.w += n * p.lw, q.sw += n;
        if (p.bias) q.bias += n;
        return q;
    }
};

// A launch holds fewer than 2^32 work-items, and the smallest tiles have 512 for
// 16 x 16 outputs: y goes in parts that stay below that with every kernel (the
// choice of one changes no bit), of whole columns where there are up to 2^15 rows.
template <typename T> hipError_t parts(const Params &p, void *ws, size_t ws_bytes, hipStream_t s)
{
    const Part part(p);
    for (long long n = 0; n < p.N; n += part.columns)
        for (long long m = 0; m < p.M; m += part.rows) {
            Params q = part.at(p, m, n);
            q.y = (T *)p.y + m * p.ly + n;
            const hipError_t e = launch<T>(q, ws, ws_bytes, s);
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

}  // namespace

// For both operands' rows, whatever their addresses turn out to be.
size_t workspace(const gconv_mm_q8_desc &d)
{
    const Params p{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, d.a_stride, d.w_stride, d.y_stride,
                   (int)d.M, (int)d.N, (int)d.K, 0, 0};
    return d.M == 0 || !pack_pays(p) ? 0 : ((size_t)d.M + (size_t)d.N) * padded(p.K);
}

hipError_t run(const gconv_mm_q8_desc &d, const int8_t *a, const float *a_scale, const int8_t *w,
               const float *w_scale, const float *bias, void *y, void *ws, size_t ws_bytes, hipStream_t s)
{
    Params p{a, w, a_scale, w_scale, bias, y, d.a_stride, d.w_stride, d.y_stride, (int)d.M, (int)d.N, (int)d.K, 0, 0};
    switch (d.dtype) {
    case GCONV_F32: return parts<float>(p, ws, ws_bytes, s);
    case GCONV_F16: return parts<_Float16>(p, ws, ws_bytes, s);
    default: return parts<__bf16>(p, ws, ws_bytes, s);
    }
}

const char *kernel(const gconv_mm_q8_desc &d, const void *a, const void *w, const void *ws, size_t ws_bytes)
{
    static const char *const names[2][kAny + 1] = {
        {"few_k 8", "few_k 16", "few_k 32", "few_k 48", "few_k 64", "tile_k 64", "tile_k 128", "tile_k 256", "few_any_k 16",
         "few_any_k 32", "few_any_k 64", "any_k"},
        {"pack_k, few_k 8", "pack_k, few_k 16", "pack_k, few_k 32", "pack_k, few_k 48", "pack_k, few_k 64",
         "pack_k, tile_k 64", "pack_k, tile_k 128", "pack_k, tile_k 256"}};
    if (d.M == 0) return "";
    const Params p{(const int8_t *)a, (const int8_t *)w, nullptr, nullptr, nullptr, nullptr, d.a_stride, d.w_stride,
                   d.y_stride, (int)d.M, (int)d.N, (int)d.K, 0, 0};
    const Route r = route(Part(p).at(p, 0, 0), ws, ws_bytes);
    return names[r.pack][r.kernel];
}

}  // namespace mmq8
}  // namespace gconv

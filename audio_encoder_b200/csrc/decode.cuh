// The attention side of one decoding step: keys and values appended to a
// paged cache with the position rotation on the way, and the attention of one
// new token per sequence over that cache.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "attn.cuh"
#include "common.cuh"
#include "gemv.cuh"

namespace moss {

enum : int { KV_BF16 = 0, KV_F16 = 1, KV_E4M3 = 2 };

// Device error word bits of the paged calls (a word of its own in the flag
// block: the bounded waits read the timeout word).
enum : int { DEV_ERR_PAGE = 1 };

// The caller's pages (moss_enc_kv_cache), with the page size as a shift.
struct PagedKV {
    uint8_t *k, *v;
    const int *table;
    long long table_stride;
    long long stride_page, stride_token, stride_head;  // bytes
    int n_seqs, pages_per_seq, n_pages, page_shift, hkv, dim;
    float k_scale, v_scale;
    int *flag;

    // Byte offset of position pos (its page already looked up).
    __device__ __forceinline__ long long at(int page, int pos) const
    {
        return page * stride_page + (pos & ((1 << page_shift) - 1)) * stride_token;
    }
    // What the table says of the page that holds position pos of sequence s
    // (0 past the table).
    __device__ __forceinline__ int entry(int s, int pos) const
    {
        return (pos >> page_shift) < pages_per_seq ? table[s * table_stride + (pos >> page_shift)] : 0;
    }
    // Whether the cache has such a page; the error word is set if not.
    __device__ __forceinline__ bool has(int page) const
    {
        if ((unsigned)page < (unsigned)n_pages) return true;
        atomicOr(flag, DEV_ERR_PAGE);
        return false;
    }
};

// ------------------------------------------------------------ append

// How rows come to the cache: as they are, as e4m3 over scales that are powers of
// two (whose reciprocals are exact), or as e4m3 over any scales.
enum : int { TO_OWN = 0, TO_E4M3_EXACT = 1, TO_E4M3 = 2 };

struct E4m3Scale {
    float scale, inv;
};

struct AppendArgs {
    PagedKV c;
    const uint16_t *k, *v, *q;
    uint16_t *q_out;
    long long k_stride, v_stride, q_stride, q_out_stride;  // elements between rows
    const int *positions, *seqs;
    const double *inv_freq;
    int n_rows, hq, rotary, interleaved;
    E4m3Scale k_scale, v_scale;
};

template <typename T>
__device__ __forceinline__ float2 to_f2(uint32_t w);
template <>
__device__ __forceinline__ float2 to_f2<bf16>(uint32_t w)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}
template <>
__device__ __forceinline__ float2 to_f2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t from_f2(float x, float y);
template <>
__device__ __forceinline__ uint32_t from_f2<bf16>(float x, float y)
{
    return pack_bf16x2(x, y);
}
template <>
__device__ __forceinline__ uint32_t from_f2<__half>(float x, float y)
{
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = to_f2<T>(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(from_f2<T>(x[0], x[1]), from_f2<T>(x[2], x[3]), from_f2<T>(x[4], x[5]), from_f2<T>(x[6], x[7]));
}

// x / scale for a rounding to e4m3, as if it were rounded once. x * inv is within 2
// ulp of the quotient; of the numbers whose last three bits are zero, all middles
// between two e4m3 values among them, the nearest is within 6, so the sign of
// what it leaves over (x - l * scale, of one multiply-add) says on which side of
// it the quotient lies, and the result is that number or its neighbour there. What
// is held at 448 anyway, and NaN, stays x * inv. (45000 rows of 16 + 8 + 8 heads x
// 128 take 131 us, 116 over powers of two; with a division, which needs the same
// step after it, 193.)
__device__ __forceinline__ float over(float x, E4m3Scale s)
{
    const float p = x * s.inv;
    const uint32_t l = (__float_as_uint(p) + 4) & ~7u;
    const float left = fmaf(-__uint_as_float(l), s.scale, x);
    const uint32_t by = left == 0.0f ? 0u : (uint32_t)((int)(__float_as_uint(left) ^ l) >> 31) | 1u;
    return fabsf(p) < 512.0f ? __uint_as_float(l + by) : p;
}

// Eight values over their scale as e4m3 (round to nearest even, held at +-448;
// NaN stays NaN).
template <int TO>
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], E4m3Scale s)
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 y = TO == TO_E4M3_EXACT ? make_float2(x[2 * i] * s.inv, x[2 * i + 1] * s.inv)
                                             : make_float2(over(x[2 * i], s), over(x[2 * i + 1], s));
        r[i] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// A CTA takes ROWS rows: an item is 16 values of each (values i .. i+7 and
// their partners, half a rotated span further, or the next eight when pairs
// lie side by side), and a thread asks for its item of all the rows before it
// looks at where they go. The rows' angles are worked out once, by all threads,
// and shared by the heads.
//
// Angles grow with the position, so they are taken in 64 bits, as a fraction
// of a turn (pos * inv_freq / 2 pi less its nearest whole number), and only
// that fraction goes to fp32 for the sine and cosine.
//
// Bound by the memory: 45000 rows of 16 + 8 + 8 heads x 128 take 121 us in a
// graph (93 % of the copy rate; 127 call by call, 88 %), four rows a CTA keeping
// 32 KB of it on the way. With one row a CTA every warp waited for positions,
// page, angles and values in turn (193 us).
template <typename T, int TO, int ROWS>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a)
{
    // cosine and sine of pair f of each row at [f % 8][f / 8]: neighbouring
    // threads have neighbouring f / 8
    __shared__ float2 cs[ROWS][128];
    __shared__ long long slots[ROWS];  // byte offset in the cache, or -1
    __shared__ int where[ROWS];
    const int tid = threadIdx.x, row0 = blockIdx.x * ROWS;
    const int per_head = a.c.dim / 16, rot_items = a.rotary / 16;
    const int items = (a.hq + 2 * a.c.hkv) * per_head;
    grid_dep_wait();
    grid_dep_launch();

    if (tid < ROWS) {
        const int row = row0 + tid;
        long long slot = -1;
        int pos = 0;
        if (row < a.n_rows) {
            const int seq = a.seqs ? a.seqs[row] : row;
            pos = a.positions[row];
            if (seq >= 0) {  // a padding row has none: nothing is written
                int page = -1;
                if (seq < a.c.n_seqs && pos >= 0 && (pos >> a.c.page_shift) < a.c.pages_per_seq) page = a.c.entry(seq, pos);
                if (a.c.has(page)) slot = a.c.at(page, pos);
            }
        }
        slots[tid] = slot;
        where[tid] = pos;
    }

    // the grid's second dimension shares out the items of few, wide rows
    bool ready = false;
    for (int it = blockIdx.y * blockDim.x + tid;; it += gridDim.y * blockDim.x) {
        const bool live = it < items;
        int h = it / per_head;
        const int j = it - h * per_head;
        const uint16_t *src = a.q;
        long long stride = a.q_stride;
        enum { Q, K, V } what = Q;
        if (h >= a.hq) {
            h -= a.hq;
            what = h < a.c.hkv ? K : V;
            h -= what == V ? a.c.hkv : 0;
            src = what == K ? a.k : a.v;
            stride = what == K ? a.k_stride : a.v_stride;
        }
        const bool turn = what != V && j < rot_items;
        const int d0 = turn && !a.interleaved ? 8 * j : 16 * j;
        const int d1 = turn && !a.interleaved ? a.rotary / 2 + 8 * j : d0 + 8;
        src += row0 * stride + h * a.c.dim;
        uint4 in[ROWS][2];
#pragma unroll
        for (int r = 0; r < ROWS; r++)
            if (live && row0 + r < a.n_rows) {
                in[r][0] = ldg_stream16(src + r * stride + d0);
                in[r][1] = ldg_stream16(src + r * stride + d1);
            }
        if (!ready) {
            ready = true;
            __syncthreads();
            for (int i = tid; i < ROWS * (a.rotary / 2); i += blockDim.x) {
                const int r = i / (a.rotary / 2), f = i - r * (a.rotary / 2);
                const double turns = (double)where[r] * a.inv_freq[f] * 0.15915494309189533577;
                const float t = (float)(turns - rint(turns));
                float s, c;
                sincospif(2.0f * t, &s, &c);
                cs[r][(f & 7) * rot_items + (f >> 3)] = make_float2(c, s);
            }
            __syncthreads();
        }
        if (!live) break;
#pragma unroll
        for (int r = 0; r < ROWS; r++) {
            const long long slot = slots[r];
            if (slot < 0) continue;
            float x[8], y[8];
            unpack8<T>(in[r][0], x);
            unpack8<T>(in[r][1], y);
            if (turn) {
                const float2 *e = cs[r] + j;
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float2 u = e[i * rot_items], w = e[(4 + i) * rot_items];
                        const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
                        x[2 * i] = x0 * u.x - x1 * u.y;
                        x[2 * i + 1] = x1 * u.x + x0 * u.y;
                        y[2 * i] = y0 * w.x - y1 * w.y;
                        y[2 * i + 1] = y1 * w.x + y0 * w.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float2 u = e[i * rot_items];
                        const float x0 = x[i], y0 = y[i];
                        x[i] = x0 * u.x - y0 * u.y;
                        y[i] = y0 * u.x + x0 * u.y;
                    }
                }
            }
            if (what == Q) {
                uint16_t *dst = a.q_out + (row0 + r) * a.q_out_stride + h * a.c.dim;
                *reinterpret_cast<uint4 *>(dst + d0) = pack8<T>(x);
                *reinterpret_cast<uint4 *>(dst + d1) = pack8<T>(y);
            } else {
                uint8_t *dst = (what == K ? a.c.k : a.c.v) + slot + h * a.c.stride_head;
                if constexpr (TO != TO_OWN) {
                    const E4m3Scale s = what == K ? a.k_scale : a.v_scale;
                    *reinterpret_cast<uint2 *>(dst + d0) = pack8_e4m3<TO>(x, s);
                    *reinterpret_cast<uint2 *>(dst + d1) = pack8_e4m3<TO>(y, s);
                } else {
                    *reinterpret_cast<uint4 *>(dst + 2 * d0) = pack8<T>(x);
                    *reinterpret_cast<uint4 *>(dst + 2 * d1) = pack8<T>(y);
                }
            }
        }
    }
}

// ------------------------------------------------------------ attention

struct PagedAttnArgs {
    PagedKV c;
    const uint16_t *q;   // [n_seqs][hq][dim], rows q_stride elements apart
    uint16_t *out;       // [n_seqs][hq][dim]
    float *lse;          // [n_seqs][hq] or null
    const int *lengths;  // [n_seqs]
    long long q_stride;
    int hq, group;       // query heads, query heads per key head
    int head_groups;     // groups of 8 NT query heads that share a key head
    bool few;            // up to 1024 sequences, whose tiles 32 bits count
    float scale_log2;    // scale * log2(e)
};

__device__ __forceinline__ void mma_16816(bf16, float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    mma_16816_bf16(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ void mma_16816(__half, float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values, rows lane / 4, columns 2 (lane % 4) and
// the next, turned over.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The lower and the upper two of four e4m3 values as f16 pairs (exact).
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t v)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t v)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint2 ldg_stream8(const void *p)
{
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// Consecutive dims of one row as they lie in the cache: 16 bytes, or the 8
// that 8 dims of an e4m3 row take.
template <int BYTES>
struct RawDims {
    uint32_t w[BYTES / 4];
    __device__ __forceinline__ void load(const uint8_t *p)
    {
        if constexpr (BYTES == 16) {
            const uint4 v = ldg_stream16(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = ldg_stream8(p);
            w[0] = v.x, w[1] = v.y;
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < BYTES / 4; i++) w[i] = 0;
    }
    // Dims 2 i and 2 i + 1 as a 16-bit pair.
    template <bool E4M3>
    __device__ __forceinline__ uint32_t pair(int i) const
    {
        return !E4M3 ? w[i] : i & 1 ? e4m3_hi(w[i >> 1]) : e4m3_lo(w[i >> 1]);
    }
};

// Dims 2 i and 2 i + 1 of two rows, turned: {row a, row b} of each dim as a
// pair. For e4m3 the bytes are paired first, which takes half the shuffles.
template <bool E4M3, int BYTES>
__device__ __forceinline__ void row_pairs(const RawDims<BYTES> &a, const RawDims<BYTES> &b, int i, uint32_t &even, uint32_t &odd)
{
    if constexpr (E4M3) {
        const uint32_t v = __byte_perm(a.w[i >> 1], b.w[i >> 1], i & 1 ? 0x7362 : 0x5140);
        even = e4m3_lo(v);
        odd = e4m3_hi(v);
    } else {
        even = __byte_perm(a.w[i], b.w[i], 0x5410);
        odd = __byte_perm(a.w[i], b.w[i], 0x7632);
    }
}

static constexpr int PA_WARPS = 8;

// Positions that a warp takes in one step, in sixteens: as many as keep 8 KB
// of the cache on its way per warp (128 KB an SM with 16 warps; with half of
// that for an e4m3 cache, 64 ragged sequences took 79 us, now 63).
__host__ __device__ constexpr int pa_sub(int dim, bool e4m3) { return dim >= 256 ? 1 : (dim == 128 ? 1 : 2) * (e4m3 ? 2 : 1); }
// Positions that the CTA's warps take at once.
__host__ __device__ constexpr int pa_tile(int dim, bool e4m3) { return 16 * PA_WARPS * pa_sub(dim, e4m3); }

// The largest 16-bit numbers below x and y (positive, or 0 or NaN, which stay).
template <typename T>
__device__ __forceinline__ uint32_t below_f2(float x, float y)
{
    const uint32_t a = __float_as_uint(x) - (x != 0.0f), b = __float_as_uint(y) - (y != 0.0f);
    if constexpr (std::is_same<T, bf16>::value) return __byte_perm(a, b, 0x7632);
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(b)), "f"(__uint_as_float(a)));
    return r;
}

// What a warp holds of up to 8 NT query heads that share a key head, over the
// positions it has seen: with s = scale log2(e) q.k, a reference m that follows
// the running maximum, l = sum 2^(s - m) and o = sum 2^(s - m) v.
//
// The reference is the maximum itself where probabilities meet the values in
// bf16, and 15 below it where they do in f16: with the largest at 2^15 (f16 ends
// at 65504) a probability down to 2^-29 of it keeps all of f16's bits and one
// down to 2^-40 some, instead of 2^-14 and 2^-25. Those that became zero would
// stay in l and be missing from o: a loss of one sign, which grows with the
// number of positions (up to 3 % of the largest's share with 2^20 of them below
// 2^-25; below 2^-40, as it is now, 2^-20).
//
// Keys and values are the A operands, straight from global memory, and the
// query heads are the 8 columns: S^T = K q^T has 16 positions x 8 heads, its
// probabilities turn into the B operands of O^T = V^T P^T by 8 x 8 transposes,
// and nothing passes through shared memory. P is the sum of two 16-bit numbers:
// the largest below the fp32 probability and what that leaves of it, rounded. So
// it is off by 2^-16 (bf16) or 2^-22 (f16) of itself, and neither part is negative
// or, from 16 bits' smallest number on, zero, which an infinite value would make
// NaN. The product with the second costs 1 to 2 % (45000 positions 37.2 -> 37.5
// us, 64 ragged e4m3 sequences 62.7 -> 63.9). Lane (g, t) reads key rows g and
// g + 8 in 16-byte pieces; which dims share an instruction's k is free as long as
// q uses the same ones.  It reads its piece g of the value rows 2t, 2t + 1,
// 2t + 8, 2t + 9 and pairs the rows' 16-bit halves, which gives the V^T operand
// with the dims in an order that only the store knows.
//
// mma.sync rather than tcgen05: a tcgen05 product has 128 rows, and its
// operands come from shared memory or TMEM; here they come straight from the
// loads, 8 columns suffice, and the reads of the cache are what bounds the
// kernel: 6.5 TB/s over 360000 positions of 8 key heads x 128 in bf16, 5.4 TB/s
// in e4m3, where a step's work is longer. Going through shared memory by cp.async
// to ask a step ahead took the former to 4.1 TB/s; holding two (smaller) steps in
// registers gained nothing in either.
template <typename T, bool E4M3, int D, int NT>
struct PagedState {
    static constexpr int KD = E4M3 ? 16 : 8;                 // dims in a lane's piece of a key row
    static constexpr int KJ = D / (4 * KD);                  // pieces
    static constexpr int VD = E4M3 && D >= 128 ? 16 : 8;     // dims in a lane's piece of a value row
    static constexpr int VI = D / (8 * VD);                  // pieces
    static constexpr int VJ = VD / 2;                        // 16-dim tiles per piece
    static constexpr int TILES = D / 16, DIM = D, COLUMNS = NT;
    static constexpr int ESZ = E4M3 ? 1 : 2;
    static constexpr int SUB = pa_sub(D, E4M3), TILE = pa_tile(D, E4M3);
    static constexpr int SLOT = NT * (TILES + 1) * 4 * 32;   // floats of a saved state
    static constexpr int BELOW = std::is_same<T, __half>::value ? 15 : 0;  // how far m is below the maximum

    uint32_t q[NT][TILES][2];
    float o[NT][TILES][4];
    float m[NT][2], l[NT][2], sc[NT][2];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int n = 0; n < NT; n++) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < TILES; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) o[n][i][j] = 0.0f;
        }
    }

    // The reference for scores up to `top`. Past 2^23 subtracting could round to
    // more than 2^16 times the largest probability, so there it is `top`.
    __device__ __forceinline__ static float below(float top)
    {
        return BELOW == 0 || !(fabsf(top) < 0x1p23f) ? top : top - BELOW;
    }

    // The query heads as B operands; heads past `heads` are zero.  An e4m3
    // cache is multiplied in f16: bf16 queries are brought to f16 by a power
    // of two of the head's own (its largest value to [256, 512)), which the
    // score's factor takes back, so no query is out of f16's range and what
    // underflows is 2^-33 of the head's largest.
    template <typename QT>
    __device__ __forceinline__ void load_q(const uint16_t *src, int heads, float scale_log2, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const bool live = n * 8 + g < heads;
            const uint16_t *p = src + (long long)(n * 8 + g) * D;
            float back = 1.0f;
            if constexpr (!E4M3) {
#pragma unroll
                for (int j = 0; j < KJ; j++) {
                    const uint4 v = live ? *reinterpret_cast<const uint4 *>(p + KD * (t + 4 * j)) : make_uint4(0, 0, 0, 0);
                    q[n][2 * j][0] = v.x, q[n][2 * j][1] = v.y, q[n][2 * j + 1][0] = v.z, q[n][2 * j + 1][1] = v.w;
                }
            } else {
                float x[KJ][16];
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < KJ; j++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const uint4 v = live ? *reinterpret_cast<const uint4 *>(p + KD * (t + 4 * j) + 8 * i) : make_uint4(0, 0, 0, 0);
                        unpack8<QT>(v, *reinterpret_cast<float(*)[8]>(&x[j][8 * i]));
#pragma unroll
                        for (int e = 0; e < 8; e++) top = fmaxf(top, fabsf(x[j][8 * i + e]));
                    }
                float up = 1.0f;
                if constexpr (!std::is_same<QT, __half>::value) {
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    if (top > 0.0f && top < INFINITY) {
                        const int e = min(max(8 - ilogbf(top), -126), 126);
                        up = ldexpf(1.0f, e);
                        back = ldexpf(1.0f, -e);
                    }
                }
#pragma unroll
                for (int j = 0; j < KJ; j++)
#pragma unroll
                    for (int s = 0; s < 4; s++)
#pragma unroll
                        for (int e = 0; e < 2; e++)
                            q[n][4 * j + s][e] = from_f2<__half>(x[j][4 * s + 2 * e] * up, x[j][4 * s + 2 * e + 1] * up);
            }
            // the factor of head 2t (and the next), from the lanes that hold its query
            sc[n][0] = scale_log2 * __shfl_sync(0xFFFFFFFFu, back, 8 * t);
            sc[n][1] = scale_log2 * __shfl_sync(0xFFFFFFFFu, back, 8 * t + 4);
        }
    }

    // Positions p0 .. p0 + 16 SUB - 1, those at or past `end` masked. off[i]:
    // where position p0 + 16 i lies (sixteen positions share a page), or one
    // before it when that is past the end.
    __device__ __forceinline__ void step(const PagedKV &c, const long long (&off)[SUB], int p0, int end, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
        RawDims<16> k[SUB][2][KJ];
        RawDims<VD * ESZ> v[SUB][VI][4];
#pragma unroll
        for (int u = 0; u < SUB; u++) {
            const uint8_t *p = c.k + off[u] + g * c.stride_token + t * 16;
#pragma unroll
            for (int j = 0; j < KJ; j++) {
                k[u][0][j].load(p + 64 * j);
                k[u][1][j].load(p + 8 * c.stride_token + 64 * j);
            }
        }
#pragma unroll
        for (int u = 0; u < SUB; u++) {
            const uint8_t *p = c.v + off[u] + 2 * t * c.stride_token + g * VD * ESZ;
#pragma unroll
            for (int i = 0; i < VI; i++) {
                v[u][i][0].load(p + i * 8 * VD * ESZ);
                v[u][i][1].load(p + i * 8 * VD * ESZ + c.stride_token);
                v[u][i][2].load(p + i * 8 * VD * ESZ + 8 * c.stride_token);
                v[u][i][3].load(p + i * 8 * VD * ESZ + 9 * c.stride_token);
            }
        }
        uint32_t pb[SUB][NT][2], pr[SUB][NT][2];  // the probabilities' two parts
        float s[SUB][NT][4];
#pragma unroll
        for (int u = 0; u < SUB; u++) {
#pragma unroll
            for (int n = 0; n < NT; n++) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.0f;
#pragma unroll
            for (int j = 0; j < KJ; j++)
#pragma unroll
                for (int e = 0; e < KD / 4; e++) {
                    const uint32_t a0 = k[u][0][j].template pair<E4M3>(2 * e), a1 = k[u][1][j].template pair<E4M3>(2 * e);
                    const uint32_t a2 = k[u][0][j].template pair<E4M3>(2 * e + 1), a3 = k[u][1][j].template pair<E4M3>(2 * e + 1);
#pragma unroll
                    for (int n = 0; n < NT; n++)
                        mma_16816(T(), s[u][n], a0, a1, a2, a3, q[n][j * (KD / 4) + e][0], q[n][j * (KD / 4) + e][1]);
                }
        }
#pragma unroll
        for (int n = 0; n < NT; n++) {
            // positions g (0, 1) and g + 8 (2, 3) of each sixteen, heads 2t and 2t + 1
            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
            for (int u = 0; u < SUB; u++) {
                const bool lo = p0 + 16 * u + g < end, hi = p0 + 16 * u + g + 8 < end;
                s[u][n][0] = lo ? s[u][n][0] * sc[n][0] : -INFINITY;
                s[u][n][1] = lo ? s[u][n][1] * sc[n][1] : -INFINITY;
                s[u][n][2] = hi ? s[u][n][2] * sc[n][0] : -INFINITY;
                s[u][n][3] = hi ? s[u][n][3] * sc[n][1] : -INFINITY;
                t0 = fmaxf(t0, fmaxf(s[u][n][0], s[u][n][2]));
                t1 = fmaxf(t1, fmaxf(s[u][n][1], s[u][n][3]));
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, x));
                t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, x));
            }
            t0 = below(t0), t1 = below(t1);
            if (__any_sync(0xFFFFFFFFu, t0 > m[n][0] || t1 > m[n][1])) {
                const float n0 = fmaxf(m[n][0], t0), n1 = fmaxf(m[n][1], t1);
                const float f0 = n0 == -INFINITY ? 1.0f : ex2_approx(m[n][0] - n0);
                const float f1 = n1 == -INFINITY ? 1.0f : ex2_approx(m[n][1] - n1);
                m[n][0] = n0, m[n][1] = n1;
                l[n][0] *= f0, l[n][1] *= f1;
#pragma unroll
                for (int i = 0; i < TILES; i++) {
                    o[n][i][0] *= f0, o[n][i][1] *= f1, o[n][i][2] *= f0, o[n][i][3] *= f1;
                }
            }
            const float b0 = m[n][0] == -INFINITY ? 0.0f : m[n][0], b1 = m[n][1] == -INFINITY ? 0.0f : m[n][1];
#pragma unroll
            for (int u = 0; u < SUB; u++) {
                const float e0 = ex2_approx(s[u][n][0] - b0), e1 = ex2_approx(s[u][n][1] - b1);
                const float e2 = ex2_approx(s[u][n][2] - b0), e3 = ex2_approx(s[u][n][3] - b1);
                l[n][0] += e0 + e2, l[n][1] += e1 + e3;
                const uint32_t lo = below_f2<T>(e0, e1), hi = below_f2<T>(e2, e3);
                const float2 flo = to_f2<T>(lo), fhi = to_f2<T>(hi);
                pb[u][n][0] = movmatrix(lo);
                pb[u][n][1] = movmatrix(hi);
                pr[u][n][0] = movmatrix(from_f2<T>(e0 - flo.x, e1 - flo.y));
                pr[u][n][1] = movmatrix(from_f2<T>(e2 - fhi.x, e3 - fhi.y));
            }
        }
        if (p0 + 16 * SUB > end) {
            // masked rows hold anything: 0 * NaN must not reach the sum
#pragma unroll
            for (int u = 0; u < SUB; u++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    if (p0 + 16 * u + 2 * t + (r & 1) + 4 * (r & 2) >= end)
#pragma unroll
                        for (int i = 0; i < VI; i++) v[u][i][r].zero();
        }
#pragma unroll
        for (int u = 0; u < SUB; u++)
#pragma unroll
            for (int i = 0; i < VI; i++)
#pragma unroll
                for (int j = 0; j < VJ; j++) {
                    uint32_t a0, a1, a2, a3;
                    row_pairs<E4M3>(v[u][i][0], v[u][i][1], j, a0, a1);
                    row_pairs<E4M3>(v[u][i][2], v[u][i][3], j, a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        mma_16816(T(), o[n][i * VJ + j], a0, a1, a2, a3, pb[u][n][0], pb[u][n][1]);
                        mma_16816(T(), o[n][i * VJ + j], a0, a1, a2, a3, pr[u][n][0], pr[u][n][1]);
                    }
                }
    }

    // The table's entries for a step at p0. They may be asked for before the
    // sequence's length is known; what lies past it is not looked at.
    __device__ __forceinline__ static void pages(const PagedKV &c, int s, int p0, int (&page)[SUB])
    {
#pragma unroll
        for (int u = 0; u < SUB; u++) page[u] = c.entry(s, p0 + 16 * u);
    }

    // Positions p0, p0 + stride, ... below `end`, a step at each, of one key
    // head of sequence s; `page`: the table's entries for the first. Each
    // step's entries are read a step ahead.
    __device__ __forceinline__ void run(const PagedKV &c, int s, int head, int p0, int stride, int end, int (&page)[SUB], int lane)
    {
        while (p0 < end) {
            long long off[SUB];
#pragma unroll
            for (int u = 0; u < SUB; u++) {
                if (u == 0 || p0 + 16 * u < end)
                    off[u] = c.at(c.has(page[u]) ? page[u] : 0, p0 + 16 * u) + head * c.stride_head;
                else
                    off[u] = off[u > 0 ? u - 1 : 0];
            }
            const int at = p0;
            p0 += stride;
            if (p0 < end) pages(c, s, p0, page);
            step(c, off, at, end, lane);
        }
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                l[n][0] += __shfl_xor_sync(0xFFFFFFFFu, l[n][0], x);
                l[n][1] += __shfl_xor_sync(0xFFFFFFFFu, l[n][1], x);
            }
    }

    // A state in memory: 16 bytes a lane, each column group's o tiles and then
    // its m and l.
    __device__ __forceinline__ void save(float *slot, int lane) const
    {
        float4 *p = reinterpret_cast<float4 *>(slot) + lane;
#pragma unroll
        for (int n = 0; n < NT; n++) {
#pragma unroll
            for (int i = 0; i < TILES; i++)
                p[(n * (TILES + 1) + i) * 32] = make_float4(o[n][i][0], o[n][i][1], o[n][i][2], o[n][i][3]);
            p[(n * (TILES + 1) + TILES) * 32] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
        }
    }
};

// One tile of o (16 dims of 8 query heads), with the heads' m and l.
struct PagedTile {
    float4 o, ml;

    // Tile i of column group n out of the states that slot(first), slot(first +
    // step) ... below `count` hold for different positions: eight at a time to
    // the largest maximum so far, then added in their order.
    template <class S, class F>
    __device__ __forceinline__ void gather(int n, int i, int first, int step, int count, int lane, F slot)
    {
        const int at = (n * (S::TILES + 1) + i) * 32 + lane, st = (n * (S::TILES + 1) + S::TILES) * 32 + lane;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        ml = make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
        for (; first < count; first += 8 * step) {
            float4 s[8], v[8];
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int p = first + k * step;
                s[k] = make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
                v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (p < count) {
                    const float4 *q = reinterpret_cast<const float4 *>(slot(p));
                    s[k] = q[st], v[k] = q[at];
                }
            }
            float m0 = ml.x, m1 = ml.y;
#pragma unroll
            for (int k = 0; k < 8; k++) m0 = fmaxf(m0, s[k].x), m1 = fmaxf(m1, s[k].y);
            const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
            const float f0 = ex2_approx(ml.x - b0), f1 = ex2_approx(ml.y - b1);
            ml = make_float4(m0, m1, ml.z * f0, ml.w * f1);
            o = make_float4(o.x * f0, o.y * f1, o.z * f0, o.w * f1);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float e0 = ex2_approx(s[k].x - b0), e1 = ex2_approx(s[k].y - b1);
                ml.z += s[k].z * e0, ml.w += s[k].w * e1;
                o.x += v[k].x * e0, o.y += v[k].y * e1, o.z += v[k].z * e0, o.w += v[k].w * e1;
            }
        }
    }

    // The tile to its place in a saved state.
    template <class S>
    __device__ __forceinline__ void save(float *slot, int n, int i, int lane) const
    {
        float4 *p = reinterpret_cast<float4 *>(slot) + lane;
        p[(n * (S::TILES + 1) + i) * 32] = o;
        if (i == 0) p[(n * (S::TILES + 1) + S::TILES) * 32] = ml;
    }

    // The tile's part of out and (tile 0) lse, of `heads` live heads.
    template <class S, typename QT>
    __device__ __forceinline__ void store(uint16_t *out, float *lse, int heads, float v_scale, int n, int i, int lane) const
    {
        const int g = lane >> 2, t = lane & 3;
        const int d = (i / S::VJ) * 8 * S::VD + g * S::VD + 2 * (i % S::VJ);
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int h = n * 8 + 2 * t + e;
            if (h >= heads) continue;
            // in units of the maximum again (exactly), so that neither the
            // logarithm nor v_scale / l loses bits to the reference
            constexpr float DOWN = 1.0f / (1 << S::BELOW);
            const float l = (e ? ml.w : ml.z) * DOWN, inv = l == 0.0f ? 0.0f : v_scale / l;
            *reinterpret_cast<uint32_t *>(out + (long long)h * S::DIM + d) =
                from_f2<QT>((e ? o.y : o.x) * DOWN * inv, (e ? o.w : o.z) * DOWN * inv);
            if (lse && g == 0 && i == 0) lse[h] = ((e ? ml.y : ml.x) + S::BELOW + log2f(l)) * 0.69314718055994531f;
        }
    }
};

// The states of the CTA's warps through shared memory (one slot a warp), each
// warp joining its tiles: done(tile, n, i).
template <class S, class F>
__device__ __forceinline__ void warps_join(const S &st, float *slots, int warp, int lane, F done)
{
    __syncthreads();  // the slots are free
    st.save(slots + warp * S::SLOT, lane);
    __syncthreads();
    for (int x = warp; x < S::COLUMNS * S::TILES; x += PA_WARPS) {
        PagedTile t;
        t.template gather<S>(x / S::TILES, x % S::TILES, 0, 1, PA_WARPS, lane, [&](int w) { return slots + w * S::SLOT; });
        done(t, x / S::TILES, x % S::TILES);
    }
}

// The work of a launch is a row of tiles, in the order
// (sequence, key head and group of query heads, tile): the lengths are only
// known on the device, so each CTA adds them up and takes an equal share of
// the tiles. A share may end inside a unit (one sequence's key head); then the
// unit's pieces go to the workspace and paged_join_kernel puts them together,
// in the order of the positions, so results do not depend on timing. 45000
// positions of 8 key heads x 128: 38 us (580 with a CTA per unit), of which
// the reads take 28; the rest is the way to the first read and the join.

// Where a CTA's share starts.
struct PagedShare {
    long long first, count;  // tiles
    long long share;         // tiles of a full share
    int s;                   // first sequence
    long long offset;        // tiles of that sequence before the share
};

__device__ __forceinline__ int paged_len(const PagedAttnArgs &a, int s, bool report)
{
    const int cap = a.c.pages_per_seq << a.c.page_shift, len = a.lengths[s];
    if (len >= 0 && len <= cap) return len;
    if (report) atomicOr(a.c.flag, DEV_ERR_PAGE);
    return min(max(len, 0), cap);
}

// x / y of whole numbers, in 32 bits where they fit (64-bit divisions are
// long).
__device__ __forceinline__ long long quotient(long long x, long long y)
{
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

__device__ __forceinline__ PagedShare paged_part(long long total)
{
    PagedShare r;
    r.share = max(quotient(total + gridDim.x - 1, gridDim.x), 1ll);
    r.first = min(r.share * blockIdx.x, total);
    r.count = min(r.share, total - r.first);
    return r;
}

// Up to 1024 sequences, and tiles that 32 bits count: each warp by itself,
// without a barrier. Lane i adds up the tiles of its span of the sequences; the
// lanes then take one each of the span in which the share starts.
template <int TILE>
__device__ __forceinline__ PagedShare paged_share_warp(const PagedAttnArgs &a, int units)
{
    const int lane = threadIdx.x & 31, span = (a.c.n_seqs + 31) >> 5;
    const bool report = blockIdx.x == 0 && threadIdx.x < 32;
    const auto scan = [&](int v) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= d) v += o;
        }
        return v;
    };
    const auto tiles = [&](int s, bool say) {
        return s < a.c.n_seqs ? (paged_len(a, s, say) + TILE - 1) / TILE * units : 0;
    };
    PagedShare r;
    if (a.c.n_seqs == 1) {
        r = paged_part(tiles(0, report));
        r.s = 0;
        r.offset = r.first;
        return r;
    }
    int mine = 0;
    for (int i = 0; i < span; i++) mine += tiles(lane * span + i, report);
    const int upto = scan(mine);
    r = paged_part(__shfl_sync(0xFFFFFFFFu, upto, 31));
    r.s = a.c.n_seqs;
    r.offset = 0;
    const unsigned past = __ballot_sync(0xFFFFFFFFu, upto > r.first);
    if (r.count <= 0 || past == 0) return r;
    const int from = __ffs(past) - 1, before = __shfl_sync(0xFFFFFFFFu, upto - mine, from);
    if (span == 1) {
        r.s = from;
        r.offset = r.first - before;
        return r;
    }
    const int one = lane < span ? tiles(from * span + lane, false) : 0, end = before + scan(one);
    const int at = __ffs(__ballot_sync(0xFFFFFFFFu, end > r.first)) - 1;
    if (at < 0) return r;
    r.s = from * span + at;
    r.offset = r.first - __shfl_sync(0xFFFFFFFFu, end - one, at);
    return r;
}

// Thread i of the CTA's WARPS warps adds up the tiles of its span of the
// sequences; a scan over the spans gives the total and the span in which this
// CTA's share starts, whose thread walks it.
template <int TILE, int WARPS>
__device__ __forceinline__ PagedShare paged_share(const PagedAttnArgs &a, int units)
{
    if (a.few) return paged_share_warp<TILE>(a, units);
    __shared__ long long warp_sums[WARPS], found[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int span = (a.c.n_seqs + 32 * WARPS - 1) / (32 * WARPS);
    const int lo = min(tid * span, a.c.n_seqs), hi = min(lo + span, a.c.n_seqs);
    long long mine = 0;
    for (int s = lo; s < hi; s++) mine += (long long)((paged_len(a, s, blockIdx.x == 0) + TILE - 1) / TILE) * units;
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) warp_sums[warp] = upto;
    if (tid == 0) found[0] = a.c.n_seqs, found[1] = 0;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; w++) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    PagedShare r = paged_part(total);
    long long at = before + upto - mine;
    if (r.count > 0 && at <= r.first && r.first < at + mine) {
        for (int s = lo; s < hi; s++) {
            const long long t = (long long)((paged_len(a, s, false) + TILE - 1) / TILE) * units;
            if (r.first < at + t) {
                found[0] = s;
                found[1] = r.first - at;
                break;
            }
            at += t;
        }
    }
    __syncthreads();
    r.s = (int)found[0];
    r.offset = found[1];
    return r;
}

template <typename T, typename QT, bool E4M3, int D, int NT>
__global__ void __launch_bounds__(32 * PA_WARPS, D <= 128 && NT == 1 ? 2 : 1) paged_attn_kernel(PagedAttnArgs a, float *pieces)
{
    using S = PagedState<T, E4M3, D, NT>;
    extern __shared__ __align__(16) float pa_slots[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = a.c.hkv * a.head_groups;
    grid_dep_wait();
    grid_dep_launch();
    PagedShare sh = paged_share<S::TILE, PA_WARPS>(a, units);

    // sequences without a position: nobody's share
    for (int s = blockIdx.x; s < a.c.n_seqs; s += gridDim.x)
        if (paged_len(a, s, false) == 0)
            for (int i = tid; i < a.hq * (D / 8); i += 32 * PA_WARPS) {
                *reinterpret_cast<uint4 *>(a.out + (long long)s * a.hq * D + 8 * i) = make_uint4(0, 0, 0, 0);
                if (a.lse && i < a.hq) a.lse[(long long)s * a.hq + i] = -INFINITY;
            }

    S st;
    for (int s = sh.s; sh.count > 0 && s < a.c.n_seqs; s++, sh.offset = 0) {
        const int len = paged_len(a, s, false), tiles = (len + S::TILE - 1) / S::TILE;
        if (tiles == 0) continue;
        int unit = (int)quotient(sh.offset, tiles), tile = (int)(sh.offset - (long long)unit * tiles);
        for (; unit < units && sh.count > 0; unit++, tile = 0) {
            const int head = unit / a.head_groups, hg = unit - head * a.head_groups;
            const int h0 = head * a.group + hg * 8 * NT, heads = min(a.group - hg * 8 * NT, 8 * NT);
            const int last = (int)min((long long)tiles, tile + sh.count);
            int page[S::SUB];
            const int p0 = tile * S::TILE + 16 * S::SUB * warp;
            S::pages(a.c, s, p0, page);
            st.clear();
            st.template load_q<QT>(a.q + s * a.q_stride + (long long)h0 * D, heads, a.scale_log2 * (E4M3 ? a.c.k_scale : 1.0f),
                                   lane);
            st.run(a.c, s, head, p0, S::TILE, min(len, last * S::TILE), page, lane);
            const bool whole = tile == 0 && last == tiles;
            float *piece = pieces + (2ll * blockIdx.x + (tile == 0)) * S::SLOT;
            warps_join(st, pa_slots, warp, lane, [&](const PagedTile &x, int n, int i) {
                if (whole)
                    x.template store<S, QT>(a.out + ((long long)s * a.hq + h0) * D, a.lse ? a.lse + (long long)s * a.hq + h0 : nullptr,
                                            heads, E4M3 ? a.c.v_scale : 1.0f, n, i, lane);
                else
                    x.template save<S>(piece, n, i, lane);
            });
            sh.count -= last - tile;
        }
    }
}

// The address of `p` (this CTA's shared memory) in the cluster's CTA `rank`.
__device__ __forceinline__ float *cluster_slot(float *p, uint32_t rank)
{
    uint64_t r;
    asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
    return reinterpret_cast<float *>(r);
}

// One cluster per unit, for lengths that a few steps of its CTAs take: they
// read its tiles in turn, and join through one another's shared memory, so
// there is neither a workspace nor a second launch. `ways`: CTAs of a cluster.
template <typename T, typename QT, bool E4M3, int D, int NT>
__global__ void __launch_bounds__(32 * PA_WARPS, D <= 128 && NT == 1 ? 2 : 1) paged_attn_unit_kernel(PagedAttnArgs a, int ways)
{
    using S = PagedState<T, E4M3, D, NT>;
    extern __shared__ __align__(16) float pa_slots[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = a.c.hkv * a.head_groups, rank = blockIdx.x % ways, which = blockIdx.x / ways;
    const int s = which / units, unit = which - s * units;
    const int head = unit / a.head_groups, hg = unit - head * a.head_groups;
    const int h0 = head * a.group + hg * 8 * NT, heads = min(a.group - hg * 8 * NT, 8 * NT);
    const int p0 = rank * S::TILE + 16 * S::SUB * warp;
    grid_dep_wait();
    grid_dep_launch();
    int page[S::SUB];
    S::pages(a.c, s, p0, page);
    const int len = paged_len(a, s, threadIdx.x == 0);
    S st;
    st.clear();
    st.template load_q<QT>(a.q + s * a.q_stride + (long long)h0 * D, heads, a.scale_log2 * (E4M3 ? a.c.k_scale : 1.0f), lane);
    st.run(a.c, s, head, p0, ways * S::TILE, len, page, lane);
    const auto store = [&](const PagedTile &x, int n, int i) {
        x.template store<S, QT>(a.out + ((long long)s * a.hq + h0) * D, a.lse ? a.lse + (long long)s * a.hq + h0 : nullptr, heads,
                                E4M3 ? a.c.v_scale : 1.0f, n, i, lane);
    };
    if (ways == 1) {
        warps_join(st, pa_slots, warp, lane, store);
        return;
    }
    float *mine = pa_slots + PA_WARPS * S::SLOT;
    warps_join(st, pa_slots, warp, lane, [&](const PagedTile &x, int n, int i) { x.template save<S>(mine, n, i, lane); });
    cluster_sync_all();
    for (int x = warp * ways + rank; x < NT * S::TILES; x += PA_WARPS * ways) {
        PagedTile t;
        t.template gather<S>(x / S::TILES, x % S::TILES, 0, 1, ways, lane, [&](int r) { return cluster_slot(mine, r); });
        store(t, x / S::TILES, x % S::TILES);
    }
    cluster_sync_all();  // nobody leaves while its slot is read
}

// One warp per unit, for many units of few positions, which leave most of a
// CTA's warps without any: no joining at all.
template <typename T, typename QT, bool E4M3, int D, int NT>
__global__ void __launch_bounds__(32 * PA_WARPS, D <= 128 && NT == 1 ? 2 : 1) paged_attn_warp_kernel(PagedAttnArgs a)
{
    using S = PagedState<T, E4M3, D, NT>;
    const int lane = threadIdx.x & 31, units = a.c.hkv * a.head_groups;
    const long long which = (long long)blockIdx.x * PA_WARPS + (threadIdx.x >> 5);
    const int s = (int)(which / units), unit = (int)(which - (long long)s * units);
    grid_dep_wait();
    grid_dep_launch();
    if (s >= a.c.n_seqs) return;
    const int head = unit / a.head_groups, hg = unit - head * a.head_groups;
    const int h0 = head * a.group + hg * 8 * NT, heads = min(a.group - hg * 8 * NT, 8 * NT);
    int page[S::SUB];
    S::pages(a.c, s, 0, page);
    const int len = paged_len(a, s, lane == 0);
    S st;
    st.clear();
    st.template load_q<QT>(a.q + s * a.q_stride + (long long)h0 * D, heads, a.scale_log2 * (E4M3 ? a.c.k_scale : 1.0f), lane);
    st.run(a.c, s, head, 0, 16 * S::SUB, len, page, lane);
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int i = 0; i < S::TILES; i++) {
            PagedTile x;
            x.o = make_float4(st.o[n][i][0], st.o[n][i][1], st.o[n][i][2], st.o[n][i][3]);
            x.ml = make_float4(st.m[n][0], st.m[n][1], st.l[n][0], st.l[n][1]);
            x.template store<S, QT>(a.out + ((long long)s * a.hq + h0) * D, a.lse ? a.lse + (long long)s * a.hq + h0 : nullptr, heads,
                                    E4M3 ? a.c.v_scale : 1.0f, n, i, lane);
        }
}

// CTA i joins the unit that was split from share i on: its first piece is the
// share's second, the others are the first pieces of the next shares. A warp
// has one tile and every PARTS-th piece. Which unit that is follows from
// the lengths, so it is worked out before the pieces are waited for (the
// lengths are older than the kernel that writes the pieces, which lets this
// one start only when they are there).
__host__ __device__ constexpr int pj_parts(int dim, int columns) { return dim * columns >= 256 ? 1 : 2; }

template <typename T, typename QT, bool E4M3, int D, int NT>
__global__ void __launch_bounds__(2 * D * NT * pj_parts(D, NT)) paged_join_kernel(PagedAttnArgs a, const float *pieces)
{
    using S = PagedState<T, E4M3, D, NT>;
    constexpr int PARTS = pj_parts(D, NT);
    __shared__ float4 part[PARTS][S::TILES * NT][2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int x = warp % (S::TILES * NT), sub = warp / (S::TILES * NT), n = x / S::TILES, i = x % S::TILES;
    const int units = a.c.hkv * a.head_groups;
    PagedShare sh = paged_share<S::TILE, S::TILES * NT * PARTS>(a, units);
    // the last unit of the share, and its tiles past the share's end
    int s = sh.s, unit = 0;
    long long left = 0;
    if (sh.count > 0 && s < a.c.n_seqs) {
        long long end = sh.offset + sh.count;  // the share's end, in tiles from sequence s's start
        int tiles;
        for (;; s++) {
            tiles = (paged_len(a, s, false) + S::TILE - 1) / S::TILE;
            if (end <= (long long)tiles * units || s + 1 >= a.c.n_seqs) break;
            end -= (long long)tiles * units;
            sh.offset -= (long long)tiles * units;
        }
        unit = tiles > 0 ? (int)quotient(end - 1, tiles) : 0;
        const long long starts = (long long)unit * tiles;
        if (starts >= sh.offset) left = starts + tiles - end;  // else it began in an earlier share
    }
    const int more = left <= 0 ? 0 : (int)min(quotient(left + sh.share - 1, sh.share), (long long)(gridDim.x - 1 - blockIdx.x));
    grid_dep_wait();
    grid_dep_launch();
    if (more <= 0) return;
    PagedTile t;
    t.template gather<S>(n, i, sub, PARTS, more + 1, lane,
                         [&](int p) { return pieces + (2ll * (blockIdx.x + p) + (p == 0)) * S::SLOT; });
    part[sub][x][0][lane] = t.o;
    part[sub][x][1][lane] = t.ml;
    __syncthreads();
    if (sub != 0) return;
    float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
    for (int p = 0; p < PARTS; p++) m0 = fmaxf(m0, part[p][x][1][lane].x), m1 = fmaxf(m1, part[p][x][1][lane].y);
    const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
    t.o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    t.ml = make_float4(m0, m1, 0.0f, 0.0f);
#pragma unroll
    for (int p = 0; p < PARTS; p++) {
        const float4 v = part[p][x][0][lane], s = part[p][x][1][lane];
        const float f0 = ex2_approx(s.x - b0), f1 = ex2_approx(s.y - b1);
        t.ml.z += s.z * f0, t.ml.w += s.w * f1;
        t.o.x += v.x * f0, t.o.y += v.y * f1, t.o.z += v.z * f0, t.o.w += v.w * f1;
    }
    const int head = unit / a.head_groups, hg = unit - head * a.head_groups;
    const int h0 = head * a.group + hg * 8 * NT, heads = min(a.group - hg * 8 * NT, 8 * NT);
    t.template store<S, QT>(a.out + ((long long)s * a.hq + h0) * D, a.lse ? a.lse + (long long)s * a.hq + h0 : nullptr, heads,
                            E4M3 ? a.c.v_scale : 1.0f, n, i, lane);
}

}  // namespace moss

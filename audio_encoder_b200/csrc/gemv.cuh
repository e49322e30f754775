// Products of a few rows (1..32) with a matrix of 4-bit codes and group
// scales, for decoding one token at a time:
//   y[m][n] = epi(sum_g s[g][n] * (sum_{k in g} x[m][k] * (c[n][k] - 8)) + b[n])
// with groups of 128 consecutive k.  Every code is read once, so the floor is
// the codes' bytes (N K / 2, plus N K / 32 of scales) at the memory's rate.
//
// The codes stay integers: c - 8 is exact in bf16, the products with x and
// their sums over a group are taken in fp32 by the tensor cores, and the fp32
// scale multiplies each group's sum once.  Nothing rounds a weight (the
// 4-bit GEMM rounds q * s to bf16, because its tiles need bf16 operands).
//
// mma.sync m16n8k16 rather than tcgen05: the weights are A (16 rows of N),
// the few rows of x are B (8 columns), and the codes go from registers into
// the instruction.  tcgen05 would need 128 expanded rows in shared memory per
// instruction, and the shared-memory writes and reads of expanded weights
// (four times the codes' bytes) would cost more than the products.
#pragma once

#include "common.cuh"

namespace moss {

enum : int { GV_BF16 = 0, GV_GELU_BF16 = 1, GV_RESID_F32 = 2, GV_F32 = 5 };  // as moss_enc_gemm's epilogues

static constexpr int GV_WARPS = 8;

struct GemvArgs {
    const bf16 *x;         // [M][K]
    const uint8_t *codes;  // [N][K/2]
    const float *scales;   // [K/128][N]
    const float *bias;     // [N] or null
    void *out;             // [M][N]
    int M, N, K, epi;
};

// d (fp32 16 x 8) += a (bf16 16 x 16) * b (bf16 16 x 8)
__device__ __forceinline__ void mma_16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes j and j + 4 of a word of eight as a bf16 pair: 0x4300 | c is 128 + c
// exactly (bf16 has 7 mantissa bits), and subtracting 136 is exact.
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int j)
{
    const uint32_t v = ((word >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 bias = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), bias);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint4 ldg_stream16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// One CTA per 16 rows of N; its warps take the groups of 128 k in turn and
// add their sums in shared memory.  A lane holds 32 consecutive codes of rows
// g and g + 8 of a group (one 16-byte load each), k = 32 t .. 32 t + 31; the
// order of k inside an instruction is free, so its k pairs are (j, j + 4) of
// each word, the pairs that one mask takes out, and x is paired the same way.
template <int MT>
__global__ void __launch_bounds__(32 * GV_WARPS) gemv_q4_kernel(GemvArgs a)
{
    __shared__ float red[GV_WARPS][MT * 8][17];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * 16;
    const int r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);
    const int groups = a.K >> 7;
    grid_dep_wait();
    grid_dep_launch();

    float acc[MT][4] = {};
    for (int kg = warp; kg < groups; kg += GV_WARPS) {
        const uint4 c0 = ldg_stream16(a.codes + (size_t)r0 * (a.K / 2) + kg * 64 + t * 16);
        const uint4 c1 = ldg_stream16(a.codes + (size_t)r1 * (a.K / 2) + kg * 64 + t * 16);
        const float s0 = a.scales[(size_t)kg * a.N + r0], s1 = a.scales[(size_t)kg * a.N + r1];
        const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
        float part[MT][4] = {};
#pragma unroll
        for (int w = 0; w < 4; w++) {
            uint32_t p0[4], p1[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                p0[j] = q4_pair(w0[w], j);
                p1[j] = q4_pair(w1[w], j);
            }
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                const int m = mt * 8 + g;
                uint4 xv = make_uint4(0, 0, 0, 0);
                if (m < a.M) xv = *reinterpret_cast<const uint4 *>(a.x + (size_t)m * a.K + kg * 128 + t * 32 + w * 8);
                // (x0, x1), (x2, x3), (x4, x5), (x6, x7) -> (x0, x4), (x1, x5), (x2, x6), (x3, x7)
                mma_16816_bf16(part[mt], p0[0], p1[0], p0[1], p1[1], __byte_perm(xv.x, xv.z, 0x5410),
                               __byte_perm(xv.x, xv.z, 0x7632));
                mma_16816_bf16(part[mt], p0[2], p1[2], p0[3], p1[3], __byte_perm(xv.y, xv.w, 0x5410),
                               __byte_perm(xv.y, xv.w, 0x7632));
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            acc[mt][0] = fmaf(part[mt][0], s0, acc[mt][0]);
            acc[mt][1] = fmaf(part[mt][1], s0, acc[mt][1]);
            acc[mt][2] = fmaf(part[mt][2], s1, acc[mt][2]);
            acc[mt][3] = fmaf(part[mt][3], s1, acc[mt][3]);
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
        red[warp][mt * 8 + 2 * t][g] = acc[mt][0];
        red[warp][mt * 8 + 2 * t + 1][g] = acc[mt][1];
        red[warp][mt * 8 + 2 * t][g + 8] = acc[mt][2];
        red[warp][mt * 8 + 2 * t + 1][g + 8] = acc[mt][3];
    }
    __syncthreads();
    for (int i = tid; i < MT * 8 * 16; i += 32 * GV_WARPS) {
        const int m = i >> 4, r = i & 15, n = n0 + r;
        if (m >= a.M || n >= a.N) continue;
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < GV_WARPS; w++) y += red[w][m][r];
        if (a.bias) y += a.bias[n];
        const size_t o = (size_t)m * a.N + n;
        if (a.epi == GV_F32)
            static_cast<float *>(a.out)[o] = y;
        else if (a.epi == GV_RESID_F32)
            static_cast<float *>(a.out)[o] += y;
        else
            static_cast<bf16 *>(a.out)[o] = __float2bfloat16(a.epi == GV_GELU_BF16 ? gelu_fast(y) : y);
    }
}

}  // namespace moss

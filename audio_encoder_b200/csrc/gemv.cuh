// Products of a few rows (1..32) with a matrix of 4-bit codes and group
// scales, for decoding one token at a time:
//   y[m][n] = epi(sum_g s[g][n] * (sum_{k in g} x[m][k] * (c[n][k] - 8)) + b[n])
// with groups of 128 consecutive k.  Every code is read once, so the floor is
// the codes' bytes (N K / 2, plus N K / 32 of scales) at the memory's rate.
//
// The codes go to the tensor cores as they are: masked out of their word, a
// pair of codes c in the low byte of each half is the bf16 pair c * 2^-133 (or
// 16 c * 2^-133), because the first two binades of a binary format are linear
// in its bits. So a pair costs one AND and every second one half a shift, no
// conversion and no subtraction (adding 128 to make normal numbers, and taking
// 136 off, cost twice the integer instructions: 45.4 us for 8 x 131071 x 2048).
// x is multiplied by 2^90 (and by 2^-4 where it meets 16 c), which is exact, and
// a group's sum starts from -8 times the group's sum of x:
//   sum (c - 8) x = -8 sum x + sum c x.
// A group's sum is fp32, and its fp32 scale multiplies it once: nothing rounds
// a weight (the 4-bit GEMM rounds q * s to bf16, because its tiles need bf16
// operands). What is held is 2^-43 of the products and sums until the end, so
// they are normal fp32 numbers from 2^-83 on, and below it steps of 2^-106; the
// sum of a group of x is held as it is, so it has to stay below 2^128. An
// infinity in a row of x makes that row NaN.
//
// mma.sync m16n8k16: the weights are A (16 rows of N), the few rows of x are B
// (8 columns), and the codes go from registers into the instruction. tcgen05
// takes 128 rows of N at a time, with the expanded codes (four times the codes'
// bytes) in shared memory or in TMEM; the latter was not tried here, and could
// serve 9 to 32 rows, where each sixteen rows of N now read all of x from shared
// memory.
#pragma once

#include "common.cuh"

namespace moss {

enum : int { GV_BF16 = 0, GV_GELU_BF16 = 1, GV_RESID_F32 = 2, GV_F32 = 5 };  // as moss_enc_gemm's epilogues

// Groups of codes that a warp has on the way: 4 KB of 16 or 32 rows.
__host__ __device__ constexpr int gv_depth(int rt) { return 4 / rt; }

struct GemvArgs {
    const bf16 *x;         // [M][K]
    const uint8_t *codes;  // [N][K/2]
    const float *scales;   // [K/128][N]
    const float *bias;     // [N] or null
    void *out;             // [M][N]
    int M, N, K, epi;
    int split;    // warps that share a row tile's groups
    int k_stage;  // k of x that shared memory holds at a time
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

// Codes j and j + 4 of a word of eight, times 1 (even j) or 16 (odd j), as the
// bf16 pair of that multiple of 2^-133.
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int j)
{
    return (j < 2 ? word : word >> 8) & (j & 1 ? 0x00F000F0u : 0x000F000Fu);
}

__device__ __forceinline__ uint4 ldg_stream16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The warps' sums, in two buffers.
__host__ __device__ constexpr size_t gv_red_bytes(int mt, int rt, int warps)
{
    return sizeof(float) * 2 * warps * mt * 8 * (16 * rt + 1);
}
// Shared memory of k values of M rows of x: themselves, and a sum and a factor
// per group.
__host__ __device__ constexpr size_t gv_x_bytes(int mt, int M, long long k) { return 2 * (size_t)M * k + mt * 64 * (size_t)(k / 128); }

// Persistent CTAs of WARPS warps. A row tile is 16 RT rows of N; `split` warps
// share one, taking its groups of 128 k in turn, and add their sums in shared
// memory; the CTA's WARPS / split row tiles make its tile.
//
// A lane holds 32 consecutive codes of rows g and g + 8 of a group (one 16-byte
// load each), k = 32 t .. 32 t + 31; the order of k inside an instruction is
// free, so its k pairs are (j, j + 4) of each word, the pairs that one mask
// takes out, and x is paired the same way when it is put into shared memory,
// in the order in which the lanes read it. Codes are asked for DEPTH groups
// ahead, across tiles: 4 KB a warp, 64 KB an SM. (Reading x through the
// first-level cache instead, in its own order, used up that cache's rate: 8 x
// 131071 x 2048 took 52.7 us.)
//
// The reads do not bound it: these reads alone (16 rows x 64 bytes a warp and
// group) take 23 us for 131072 x 2048, as a copy does, and the kernel takes 35 us
// for 8 rows (64 % of the copy rate). No unit is full either (49 % of the issue
// slots, 23 % of the tensor pipe): 16 warps an SM wait for their loads and for one
// instruction after the other. 32 rows a warp share what 8 rows of x cost (37.2
// us with 16); a queue in shared memory filled by cp.async (37.2), 24 warps an SM
// (38.5) and requests of 256 bytes a row (37.4) gained nothing.
//
// The order of the sums depends on N, K and the number of SMs alone, so a row
// of x gives the same bits whatever other rows are with it.
template <int MT, int RT, int WARPS, bool STAGED>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) gemv_q4_kernel(GemvArgs a)
{
    constexpr int ROWS = 16 * RT, DEPTH = gv_depth(RT);
    extern __shared__ __align__(16) uint8_t gv_smem[];
    float(*red)[MT * 8][ROWS + 1] = reinterpret_cast<float(*)[MT * 8][ROWS + 1]>(gv_smem);  // [2 WARPS]
    float *xsum = reinterpret_cast<float *>(gv_smem + gv_red_bytes(MT, RT, WARPS));  // [k / 128][MT * 8]
    float *xshort = xsum + MT * 8 * (min(a.k_stage, a.K) >> 7);                  // the same
    uint4 *xs = reinterpret_cast<uint4 *>(xshort + MT * 8 * (min(a.k_stage, a.K) >> 7));  // [k / 128][word][M][t]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int split = a.split, wk = warp % split, wn = warp / split, per_cta = WARPS / split;
    const int groups = a.K >> 7, row_tiles = (a.N + ROWS - 1) / ROWS, cta_tiles = (row_tiles + per_cta - 1) / per_cta;
    const size_t row_bytes = (size_t)a.K / 2;

    struct Item {
        uint4 c[2 * RT];
        float s[2 * RT];
    } item[DEPTH];
    // Where this lane's codes and scales of a row tile lie, rows g, g + 8, ...
    // (rows past the last are the last one), and how far its next group is.
    const uint8_t *code[2 * RT];
    const float *scale[2 * RT];
    const size_t c_step = (size_t)split * 64, s_step = (size_t)split * a.N;
    const auto point = [&](int tile, int kg) {
        const long long n = (long long)(tile * per_cta + wn) * ROWS + g;
#pragma unroll
        for (int i = 0; i < 2 * RT; i++) {
            const long long r = min(n + 8 * i, (long long)a.N - 1);
            code[i] = a.codes + r * row_bytes + kg * 64 + t * 16;
            scale[i] = a.scales + (size_t)kg * a.N + r;
        }
    };
    const auto fetch = [&](Item &x) {
#pragma unroll
        for (int i = 0; i < 2 * RT; i++) {
            x.c[i] = ldg_stream16(code[i]);
            x.s[i] = *scale[i];
            code[i] += c_step, scale[i] += s_step;
        }
    };
    // x for k of [k0, k0 + n), scaled, in pairs (x0, x4), (x1, x5) / 16, (x2,
    // x6), (x3, x7) / 16, and the groups' sums; a thread has 32 values of a row.
    // A group with a value of 2^36 or more, which 2^90 times itself might not
    // hold, is not scaled, and says by which factor its sums fall short.
    bool huge = false;  // whether any group is such a one
    const auto stage = [&](int k0, int n) {
        bool mine = false;
        // four neighbours have a row's group; a round is 8 WARPS of them
        const int tt = tid & 3, m_step = 8 * WARPS % a.M, kg_step = 8 * WARPS / a.M;
        for (int m = (tid >> 2) % a.M, kg = (tid >> 2) / a.M; kg < n >> 7;) {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.x + (size_t)m * a.K + k0 + kg * 128 + tt * 32);
            uint4 in[4];
#pragma unroll
            for (int w = 0; w < 4; w++) in[w] = src[w];
            float sum = 0.0f;
            __nv_bfloat162 most = __float2bfloat162_rn(0.0f);
#pragma unroll
            for (int w = 0; w < 4; w++) {
                const uint32_t p[4] = {in[w].x, in[w].y, in[w].z, in[w].w};
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&p[j]);
                    const float2 f = __bfloat1622float2(v);
                    sum += f.x + f.y;
                    most = __hmax2(most, __habs2(v));
                }
            }
            float top = fmaxf(__low2float(most), __high2float(most));
            // a row's four threads are neighbours, and all here
            const uint32_t four = 0xFu << (lane & 28);
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                sum += __shfl_xor_sync(four, sum, d);
                top = fmaxf(top, __shfl_xor_sync(four, top, d));
            }
            const bool big = top >= 0x1p36f;
            mine |= big;
            const float up = big ? 1.0f : 0x1p90f;
            const __nv_bfloat162 u1 = __float2bfloat162_rn(up), u16 = __float2bfloat162_rn(up * 0.0625f);
#pragma unroll
            for (int w = 0; w < 4; w++) {
                uint32_t p[4] = {__byte_perm(in[w].x, in[w].z, 0x5410), __byte_perm(in[w].x, in[w].z, 0x7632),
                                 __byte_perm(in[w].y, in[w].w, 0x5410), __byte_perm(in[w].y, in[w].w, 0x7632)};
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&p[j]), j & 1 ? u16 : u1);
                    p[j] = *reinterpret_cast<const uint32_t *>(&v);
                }
                xs[((kg * 4 + w) * a.M + m) * 4 + tt] = make_uint4(p[0], p[1], p[2], p[3]);
            }
            if (tt == 0) {
                xsum[kg * MT * 8 + m] = sum * (-8.0f * 0x1p-43f) * (up * 0x1p-90f);
                xshort[kg * MT * 8 + m] = big ? 0x1p90f : 1.0f;
            }
            m += m_step, kg += kg_step;
            if (m >= a.M) m -= a.M, kg++;
        }
        huge = __syncthreads_or(mine);
    };
    int col[MT];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) col[mt] = min(mt * 8 + g, a.M - 1) * 4 + t;
    float acc[RT][MT][4];
    const auto clear = [&] {
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int mt = 0; mt < MT; mt++) acc[r][mt][0] = acc[r][mt][1] = acc[r][mt][2] = acc[r][mt][3] = 0.0f;
    };
    // a group's products; at: the group's place in xs. The sums stay 2^(90 -
    // 133) of themselves until the end.
    const auto take = [&](const Item &x, int at) {
        const uint4 *xg = xs + (size_t)at * 16 * a.M;
        float part[RT][MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            const float2 b = *reinterpret_cast<const float2 *>(xsum + (at * MT + mt) * 8 + 2 * t);
#pragma unroll
            for (int r = 0; r < RT; r++) {
                part[r][mt][0] = part[r][mt][2] = b.x;
                part[r][mt][1] = part[r][mt][3] = b.y;
            }
        }
#pragma unroll
        for (int w = 0; w < 4; w++) {
            uint32_t c[2 * RT][4];
#pragma unroll
            for (int i = 0; i < 2 * RT; i++) {
                const uint32_t word = w == 0 ? x.c[i].x : w == 1 ? x.c[i].y : w == 2 ? x.c[i].z : x.c[i].w;
#pragma unroll
                for (int j = 0; j < 4; j++) c[i][j] = q4_pair(word, j);
            }
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                // columns past the last row repeat it; nobody reads their sums
                const uint4 xv = xg[w * a.M * 4 + col[mt]];
#pragma unroll
                for (int r = 0; r < RT; r++)
                    mma_16816_bf16(part[r][mt], c[2 * r][0], c[2 * r + 1][0], c[2 * r][1], c[2 * r + 1][1], xv.x, xv.y);
#pragma unroll
                for (int r = 0; r < RT; r++)
                    mma_16816_bf16(part[r][mt], c[2 * r][2], c[2 * r + 1][2], c[2 * r][3], c[2 * r + 1][3], xv.z, xv.w);
            }
        }
        if (huge)
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                const float2 f = *reinterpret_cast<const float2 *>(xshort + (at * MT + mt) * 8 + 2 * t);
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    part[r][mt][0] *= f.x, part[r][mt][1] *= f.y, part[r][mt][2] *= f.x, part[r][mt][3] *= f.y;
                }
            }
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                acc[r][mt][0] = fmaf(part[r][mt][0], x.s[2 * r], acc[r][mt][0]);
                acc[r][mt][1] = fmaf(part[r][mt][1], x.s[2 * r], acc[r][mt][1]);
                acc[r][mt][2] = fmaf(part[r][mt][2], x.s[2 * r + 1], acc[r][mt][2]);
                acc[r][mt][3] = fmaf(part[r][mt][3], x.s[2 * r + 1], acc[r][mt][3]);
            }
    };
    // The bias of this lane's column of the outputs (all its outputs of a tile
    // have the same), asked for when the tile begins.
    float bias = 0.0f;
    const auto begin = [&](int tile) {
        const long long n = (long long)(tile * per_cta + wn) * ROWS + lane % ROWS;
        if (a.bias && tile < cta_tiles && n < a.N) bias = a.bias[n];
    };
    // The sums of the row tile's warps, who wait for one another alone, and the
    // epilogue. With two buffers one barrier a tile is enough.
    int buf = 0;
    const auto finish = [&](int tile) {
        float(*mine)[ROWS + 1] = red[buf * WARPS + warp];
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                mine[mt * 8 + 2 * t][16 * r + g] = acc[r][mt][0];
                mine[mt * 8 + 2 * t + 1][16 * r + g] = acc[r][mt][1];
                mine[mt * 8 + 2 * t][16 * r + g + 8] = acc[r][mt][2];
                mine[mt * 8 + 2 * t + 1][16 * r + g + 8] = acc[r][mt][3];
            }
        if (split > 1)
            named_bar_sync(1 + wn, 32 * split);
        else
            __syncwarp();
        const int r = lane % ROWS;
        const long long n = (long long)(tile * per_cta + wn) * ROWS + r;
        if (n < a.N)
            for (int m = wk * (32 / ROWS) + lane / ROWS; m < a.M; m += split * (32 / ROWS)) {
                float y = 0.0f;
                for (int w = 0; w < split; w++) y += red[buf * WARPS + wn * split + w][m][r];
                y = y * 0x1p43f + bias;
                const size_t o = (size_t)m * a.N + n;
                if (a.epi == GV_F32)
                    static_cast<float *>(a.out)[o] = y;
                else if (a.epi == GV_RESID_F32)
                    static_cast<float *>(a.out)[o] += y;
                else
                    static_cast<bf16 *>(a.out)[o] = __float2bfloat16(a.epi == GV_GELU_BF16 ? gelu_fast(y) : y);
            }
        buf ^= 1;
        clear();
        begin(tile + gridDim.x);
    };
    grid_dep_wait();
    grid_dep_launch();
    clear();
    begin(blockIdx.x);
    if constexpr (STAGED) {
        for (int tile = blockIdx.x; tile < cta_tiles; tile += gridDim.x) {
            for (int k0 = 0; k0 < a.K; k0 += a.k_stage) {
                const int n = min(a.k_stage, a.K - k0) >> 7;
                __syncthreads();
                stage(k0, 128 * n);
                point(tile, (k0 >> 7) + wk);
                for (int kg = wk; kg < n; kg += DEPTH * split) {
#pragma unroll
                    for (int d = 0; d < DEPTH; d++)
                        if (kg + d * split < n) fetch(item[d]);
#pragma unroll
                    for (int d = 0; d < DEPTH; d++)
                        if (kg + d * split < n) take(item[d], kg + d * split);
                }
            }
            finish(tile);
        }
    } else {
        int next_tile = blockIdx.x, next_kg = wk;  // what is asked for next
        // Not under a condition (past the last tile it is asked for again): the
        // registers of a conditional load are waited for where the cases meet.
        const auto ask = [&](Item &x) {
            fetch(x);
            next_kg += split;
            if (next_kg >= groups) {
                next_kg = wk;
                next_tile = min(next_tile + (int)gridDim.x, cta_tiles - 1);
                point(next_tile, wk);
            }
        };
        point(next_tile, wk);
#pragma unroll
        for (int d = 0; d < DEPTH; d++) ask(item[d]);
        stage(0, a.K);
        int tile = blockIdx.x, kg = wk;
        while (tile < cta_tiles) {
#pragma unroll
            for (int d = 0; d < DEPTH; d++) {
                if (tile >= cta_tiles) break;
                take(item[d], kg);
                ask(item[d]);
                kg += split;
                if (kg >= groups) {
                    finish(tile);
                    kg = wk;
                    tile += gridDim.x;
                }
            }
        }
    }
}

}  // namespace moss

// ep_expert_gemm.hip -- the experts' products on the grouped rows: E4M3 codes with a scale for each
// block of 128 on matrix cores (gfx950).  Definitions in ep_experts.h.
//
// out[m][c] = sum over blocks b of sx[m][b] sw[c / 128][b] * (x[m] . w[c] over block b).  One
// v_mfma_f32_16x16x128_f8f6f4 covers exactly one block of 128 channels, so each takes a zero
// accumulator and its 16 x 16 result is scaled into the f32 sums by ordinary fused multiply-adds
// (the instruction's own scales are powers of two and cannot hold these).  The weights are the A
// operand and the rows the B operand, so a lane's four results are four neighbouring columns of one
// row: one scale a lane and contiguous stores.
#include <limits.h>

#include "ep_experts_internal.h"

namespace ep {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// What a block works on: rows [first, first + rows) of the grouped rows, all of expert `expert`.
struct Tile {
    int expert;
    int rows;  // 0: nothing to do
    int64_t first;
};

// Tile `index` of the row tiles of all segments, in segment order, bm rows each.  Every wave finds
// it for itself: a scan over the segment sizes, 64 experts at a time.
__device__ __forceinline__ Tile find_tile(const GemmArgs &p, int bm, int index, bool report) {
    Tile t = {0, 0, 0};
    if (p.expert_rows == nullptr) {
        t.first = (int64_t)index * bm;
        const int64_t left = p.num_rows - t.first;
        t.rows = left <= 0 ? 0 : left < bm ? (int)left : bm;
        return t;
    }
    const int lane = threadIdx.x & (kWave - 1);
    int64_t rows_before = 0;
    int tiles_before = 0;
    bool found = false;
    for (int e0 = 0; e0 < p.num_experts; e0 += kWave) {
        int size = 0;
        if (e0 + lane < p.num_experts) size = p.expert_rows[e0 + lane];
        if (size < 0) size = 0;
        const int64_t end = rows_before + wave_inclusive_scan64(size), start = end - size;
        int64_t fit = p.num_rows - start;  // rows of the segment that are inside the buffers
        fit = fit < 0 ? 0 : fit < size ? fit : size;
        const int tiles = (int)((fit + bm - 1) / bm);
        const int upto = tiles_before + wave_inclusive_scan(tiles);
        const uint64_t past = ballot64(upto > index);
        if (!found && past != 0ull) {
            const int l = __builtin_ctzll(past);
            const int64_t skip = (int64_t)(index - readlane32(upto - tiles, l)) * bm;
            const int64_t rows = (int64_t)readlane64((uint64_t)fit, l) - skip;
            t.expert = e0 + l;
            t.first = (int64_t)readlane64((uint64_t)start, l) + skip;
            t.rows = rows < bm ? (int)rows : bm;
            found = true;
            if (!report) return t;
        }
        rows_before = (int64_t)readlane64((uint64_t)end, kWave - 1);
        tiles_before = readlane32(upto, kWave - 1);
    }
    if (report && rows_before > p.num_rows && threadIdx.x == 0) flag(p.dev_status, EP_DEV_RECV_OVERFLOW);
    return t;
}

constexpr int kBM = 128, kBN = 256, kThreads = 256;
constexpr int kUnits = kScaleBlock / 16;  // 16-byte units of a row in one block of channels

// LDS place of unit c of row r: rotating the units by the row spreads the 16 rows that a wave reads
// at once over all banks.
__device__ __forceinline__ int place(int r, int c) { return r * kUnits + (c ^ (r & (kUnits - 1))); }

// kBM rows x kBN weight rows a block, 2 x 2 waves of 64 x 128.  SWIGLU: each wave's 128 weight rows
// are 64 gate rows and the 64 up rows of the same outputs.
template <bool SWIGLU>
__global__ __launch_bounds__(kThreads) void expert_gemm_kernel(GemmArgs p, int col_tiles) {
    __shared__ u32x4 s_x[kBM * kUnits];
    __shared__ u32x4 s_w[kBN * kUnits];
    __shared__ float s_top[2][kBM];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int col_tile = blockIdx.x % col_tiles;
    const Tile t = find_tile(p, kBM, blockIdx.x / col_tiles, blockIdx.x == 0);
    if (t.rows == 0) return;  // the whole block: every wave found the same
    const int wrows = SWIGLU ? 2 * p.n : p.n;  // weight rows of an expert
    const int blocks = p.k / kScaleBlock;
    const int scale_rows = (wrows + kScaleBlock - 1) / kScaleBlock;
    const uint8_t *x = p.x + t.first * p.k;
    const uint8_t *w = p.w + (int64_t)t.expert * wrows * p.k;
    const float *sx = p.x_scales + t.first * blocks;
    const float *sw = p.w_scales + (int64_t)t.expert * scale_rows * blocks;

    // weight row behind row v of the block's kBN
    auto weight_row = [&](int v) {
        if constexpr (SWIGLU) {
            const int u = v & 127, c = col_tile * 128 + (v >> 7) * 64 + (u & 63);
            return u < 64 ? c : p.n + c;
        } else {
            const int c = col_tile * kBN + v;
            return c < p.n ? c : p.n - 1;  // a column past the last is computed and not stored
        }
    };
    int scale_row0, scale_row1;  // of the wave's first and second 64 weight rows
    if constexpr (SWIGLU) {
        scale_row0 = col_tile;
        scale_row1 = p.n / kScaleBlock + col_tile;
    } else {
        scale_row0 = col_tile * (kBN / kScaleBlock) + wn;
        scale_row0 = scale_row1 = scale_row0 < scale_rows ? scale_row0 : scale_rows - 1;
    }

    constexpr int MT = 4, NT = 8;
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int q = lane >> 4, r16 = lane & 15;
    for (int b = 0; b < blocks; ++b) {
        __syncthreads();
        for (int i = threadIdx.x; i < kBM * kUnits; i += kThreads) {
            const int r = i / kUnits, c = i % kUnits;
            const int row = r < t.rows ? r : t.rows - 1;  // rows past the segment are not stored
            s_x[place(r, c)] = *reinterpret_cast<const u32x4 *>(x + (int64_t)row * p.k + b * kScaleBlock + c * 16);
        }
        for (int i = threadIdx.x; i < kBN * kUnits; i += kThreads) {
            const int r = i / kUnits, c = i % kUnits;
            s_w[place(r, c)] =
                *reinterpret_cast<const u32x4 *>(w + (int64_t)weight_row(r) * p.k + b * kScaleBlock + c * 16);
        }
        __syncthreads();
        const float sw0 = sw[(int64_t)scale_row0 * blocks + b], sw1 = sw[(int64_t)scale_row1 * blocks + b];
        auto fragment = [&](const u32x4 *s, int r) {
            const u32x4 lo = s[place(r, 2 * q)], hi = s[place(r, 2 * q + 1)];
            return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
        };
        i32x8 fx[MT];
        float scale[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = wm * 64 + i * 16 + r16;
            fx[i] = fragment(s_x, r);
            scale[i] = sx[(int64_t)(r < t.rows ? r : t.rows - 1) * blocks + b];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const i32x8 fw = fragment(s_w, wn * 128 + j * 16 + r16);
            const float swj = j < NT / 2 ? sw0 : sw1;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    fw, fx[i], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
                const float s = scale[i] * swj;
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][j][k] = __builtin_fmaf(part[k], s, acc[i][j][k]);
            }
        }
    }

    if constexpr (!SWIGLU) {
        uint32_t *out = static_cast<uint32_t *>(p.out);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = wm * 64 + i * 16 + r16;
            if (r >= t.rows) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int c = col_tile * kBN + wn * 128 + j * 16 + q * 4;
                if (c >= p.n) continue;  // n is a multiple of 8: all four or none
                uint2 o;
                o.x = pack_bf16(acc[i][j][0], acc[i][j][1]);
                o.y = pack_bf16(acc[i][j][2], acc[i][j][3]);
                *reinterpret_cast<uint2 *>(out + ((t.first + r) * p.n + c) / 2) = o;
            }
        }
    } else {
        float top[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            top[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float g = acc[i][j][k], u = acc[i][j + NT / 2][k];
                    const float a = g / (1.0f + expf(-g)) * u;
                    acc[i][j][k] = a;
                    top[i] = fmaxf(top[i], fabsf(a));
                }
            }
            top[i] = fmaxf(top[i], __shfl_xor(top[i], 16));
            top[i] = fmaxf(top[i], __shfl_xor(top[i], 32));
            if (q == 0) s_top[wn][wm * 64 + i * 16 + r16] = top[i];
        }
        __syncthreads();
        uint32_t *out = static_cast<uint32_t *>(p.out);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = wm * 64 + i * 16 + r16;
            if (r >= t.rows) continue;
            const float m = fmaxf(fmaxf(s_top[0][r], s_top[1][r]), kE4m3AmaxFloor);
            const float inv = kE4m3Max / m;
            if (wn == 0 && q == 0) p.out_scales[(t.first + r) * (p.n / kScaleBlock) + col_tile] = m / kE4m3Max;
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                const int c = col_tile * 128 + wn * 64 + j * 16 + q * 4;
                out[((t.first + r) * p.n + c) / 4] = e4m3_pack4(acc[i][j][0] * inv, acc[i][j][1] * inv,
                                                               acc[i][j][2] * inv, acc[i][j][3] * inv);
            }
        }
    }
}

int64_t row_tiles(const GemmArgs &a, int bm) {
    if (a.expert_rows == nullptr) return ((int64_t)a.num_rows + bm - 1) / bm;
    const int64_t busy = a.num_experts < a.num_rows ? a.num_experts : a.num_rows;
    return a.num_rows / bm + busy;  // each segment ends in at most one part tile
}

int64_t grid_blocks(const GemmArgs &a) {
    const int64_t cols = a.swiglu ? a.n / kScaleBlock : (a.n + kBN - 1) / kBN;
    return row_tiles(a, kBM) * cols;
}

}  // namespace

bool gemm_grid_ok(const GemmArgs &a) { return grid_blocks(a) <= INT_MAX / kThreads; }

hipError_t launch_expert_gemm(const GemmArgs &a, hipStream_t stream) {
    const int64_t blocks = grid_blocks(a);
    if (blocks == 0) return hipSuccess;
    if (a.swiglu) {
        hipLaunchKernelGGL(expert_gemm_kernel<true>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a,
                           a.n / kScaleBlock);
    } else {
        hipLaunchKernelGGL(expert_gemm_kernel<false>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a,
                           (a.n + kBN - 1) / kBN);
    }
    return hipGetLastError();
}

}  // namespace ep

// ep_expert_gemm.hip -- the experts' products on the grouped rows: E4M3 codes with a scale for each
// block of 128 on matrix cores (gfx950).  Definitions in ep_experts.h.
//
// out[m][c] = sum over blocks b of sx[m][b] sw[c / 128][b] * (x[m] . w[c] over block b).  Each block
// of 128 channels starts from a zero accumulator, and its result is scaled into the f32 sums by
// ordinary fused multiply-adds (the matrix instructions' own scales are powers of two and cannot
// hold these).  The weights are the A operand and the rows the B operand, so a lane's results are
// neighbouring columns of one row: one scale a lane and contiguous stores.
//
// The codes are turned into f16 for the f16 matrix instructions (exact: every E4M3 value is one, and a
// product of two fits f32), whose sums are f32 throughout (measured: 1e-8 of normally distributed codes'
// result).  The E4M3 instructions run at twice the rate, but add the eight products of a group of
// neighbouring channels with 13 bits below the largest one's and cut the rest of each (measured: 2^8
// keeps 2^-5 of its group and loses 2^-6): one channel at 448 * 448 would take away what its seven
// neighbours add below 24.5.
#include <limits.h>

#include "ep_experts_internal.h"

namespace ep {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

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

constexpr int kUnits = kScaleBlock / 16;  // 16-byte units of a row in one block of channels
constexpr int kBlockThreads = 512;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Half of a 16-byte unit of codes (which: 0 or 1) as one f16 operand of a 32 x 32 x 16 product.
// Every E4M3 value is an f16 value.
template <int which>
__device__ __forceinline__ f16x8 to_f16(u32x4 unit) {
    f16x8 f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int word = (int)unit[2 * which + i];
        const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, false);
        const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, true);
        f[4 * i] = a[0];
        f[4 * i + 1] = a[1];
        f[4 * i + 2] = b[0];
        f[4 * i + 3] = b[1];
    }
    return f;
}

// Buffer descriptor over `bytes` bytes from p; loads past them return 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x00027000);
}

// 64 lanes' 16-byte units from global memory straight into 1 KiB of LDS at dst (wave-uniform).
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t src, u32x4 *dst, int voffset, int soffset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void *)dst, 16, voffset, soffset,
                                             0, 0);
}

// The same for 4-byte values: 256 bytes of LDS.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t src, float *dst, int voffset, int soffset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void *)dst, 4, voffset, soffset,
                                             0, 0);
}

// Ends a step: the wave's reads of LDS are over and no more than `left` (0 .. 15) of its loads are
// under way (they end in order), and then every wave's.  __syncthreads would wait for all loads.
template <int left>
__device__ __forceinline__ void end_step() {
    static_assert(left >= 0 && left < 16, "the low bits of vmcnt");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | left);  // vmcnt(left), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Unit of row r that lies at place c of its row in LDS (and the place of unit c).  A 16-byte read
// is served 16 lanes at a time, lanes whose rows share their low three bits among them; so bits 3
// and 4 take part.
__device__ __forceinline__ int rotate(int r, int c) { return c ^ ((r ^ ((r >> 3) & 3)) & (kUnits - 1)); }

constexpr int kBN = 256;  // weight rows of a wide block

// Many rows: 64 MI rows x 256 weight rows a block, 2 x 4 waves of 32 MI rows x 64 weight rows.  A block of 128
// channels of both goes straight to LDS, two steps ahead; its products are summed by the matrix instructions and
// scaled into the wave's sums by one FMA each (a scale covers 128 channels).  The scaled sums have to be in
// registers that vector instructions reach.
//
// SwiGLU of 32768 rows of 32 experts, 7168 channels to 2048: 1875 us (median of 20; 1816 the least), 1.03 PFLOP/s;
// product of as many rows, 2048 channels to 7168: 996 us (963), 0.97.  Matrix instructions are at work in 48 to 51% of
// a SIMD's cycles and the other vector instructions (conversions, scaling) issue in 45 to 48%: the two waves of a SIMD
// leave the barrier together and convert together, so the two kinds hardly overlap.  LDS is in use for 15%, and the
// clock is at 1.95 of 2.4 GHz.  (The E4M3 instructions took the product in 606 us, without the sums' last bits.)
template <bool SWIGLU, int MI>
__global__ __launch_bounds__(kBlockThreads, 2) void expert_gemm_wide_kernel(GemmArgs p, int col_tiles) {
    constexpr int WM = 2, WN = 4, BM = 32 * MI * WM, HALF = 32;
    static_assert(2 * HALF * WN == kBN, "256 weight rows a block");
    constexpr int XL = BM * kUnits / kBlockThreads, WL = kBN * kUnits / kBlockThreads;  // units a thread loads
    // Three buffers: while one block of channels is multiplied the next two are on their way.  A
    // wave's last load of a step is of scales: rows' by the first BM lanes, the weights' two by the
    // lanes of the next wave (the others repeat those).  (One array a buffer: the compiler tells them
    // apart, and would wait for all loads before a read of an array that it does not.)
    constexpr int kLoads = XL + WL + 1;  // of a wave and step
    static_assert(BM <= 64 * (WM * WN - 1), "a wave is left for the weights' scales");
    constexpr int kX = 0, kW = BM * kUnits, kS = kW + kBN * kUnits, kBuffer = kS + kBlockThreads / 4;
    __shared__ u32x4 s_0[kBuffer], s_1[kBuffer], s_2[kBuffer];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int col_tile = blockIdx.x % col_tiles;
    const Tile t = find_tile(p, BM, blockIdx.x / col_tiles, blockIdx.x == 0);
    if (t.rows == 0) return;  // the whole block: every wave found the same
    const int wrows = SWIGLU ? 2 * p.n : p.n;
    const int blocks = p.k / kScaleBlock;
    const int scale_rows = (wrows + kScaleBlock - 1) / kScaleBlock;
    const __amdgpu_buffer_rsrc_t xbuf = descriptor(p.x + t.first * p.k, (uint32_t)t.rows * p.k);
    const __amdgpu_buffer_rsrc_t wbuf = descriptor(p.w + (int64_t)t.expert * wrows * p.k, (uint32_t)wrows * p.k);

    // where the lane's first unit of a buffer comes from; the others lie kStep rows on, each.  Units
    // go to LDS in lane order, so the rotation of a row's units is in the address they are read
    // from.  Rows past the segment, or past the last column, are past the descriptor's end: they
    // read as 0 and are not stored.
    constexpr int kStep = kBlockThreads / kUnits;
    const int r0 = threadIdx.x / kUnits, c0 = rotate(r0, threadIdx.x & (kUnits - 1)) * 16;
    static_assert(kStep % 32 == 0, "a step keeps a row's rotation");
    const uint32_t k = p.k;  // unsigned: a row past the end may lie past 2^31, and must not come out below 0
    const uint32_t x_first = r0 * k + c0;
    uint32_t w_first;
    if constexpr (SWIGLU) {
        // half of a wave's weight rows are gate rows, half the up rows of the same outputs
        static_assert(kStep % (2 * HALF) == 0, "a step keeps a row's place in its half");
        const int c = col_tile * 128 + r0 / (2 * HALF) * HALF + r0 % HALF;
        w_first = (uint32_t)((r0 & HALF) ? p.n + c : c) * k + c0;
    } else {
        w_first = (uint32_t)(col_tile * kBN + r0) * k + c0;
    }
    int scale_row0, scale_row1;  // of the first and the second 128 weight rows; gate and up
    if constexpr (SWIGLU) {
        scale_row0 = col_tile;
        scale_row1 = p.n / kScaleBlock + col_tile;
    } else {
        scale_row0 = 2 * col_tile;
        scale_row1 = 2 * col_tile + 1 < scale_rows ? 2 * col_tile + 1 : scale_rows - 1;
    }
    const __amdgpu_buffer_rsrc_t sbuf =
        wave * kWave < BM ? descriptor(p.x_scales + t.first * blocks, (uint32_t)t.rows * blocks * 4)
                          : descriptor(p.w_scales + (int64_t)t.expert * scale_rows * blocks, (uint32_t)scale_rows * blocks * 4);
    const uint32_t sat = (wave * kWave < BM ? (int)threadIdx.x : (lane & 1) ? scale_row1 : scale_row0) * blocks * 4;

    f32x16 acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    const int half = lane >> 5, r32 = lane & 31;
    const bool busy = wm * 32 * MI < t.rows;  // the other half of a part tile has nothing to multiply
    // Past the last block the loads go on, from behind the descriptors' ends (they fetch nothing):
    // that every step issues the same number is what lets the waits count.
    auto load = [&](u32x4 *to, int b) {
        const uint32_t past = b < blocks ? 0u : 0x80000000u;
        const int from = b < blocks ? b : 0;
        uint32_t xat = x_first, wat = w_first;
        asm volatile("" : "+v"(xat), "+v"(wat));  // addresses are cheaper formed anew than kept in registers
#pragma unroll
        for (int i = 0; i < XL; ++i)
            load_to_lds(xbuf, to + kX + i * kBlockThreads + wave * kWave, (int)(xat + (i * kStep * k + past)), from * kScaleBlock);
#pragma unroll
        for (int i = 0; i < WL; ++i)
            load_to_lds(wbuf, to + kW + i * kBlockThreads + wave * kWave,
                        (int)(wat + (i * (SWIGLU ? kStep / 2 : kStep) * k + past)), from * kScaleBlock);
        load_to_lds(sbuf, reinterpret_cast<float *>(to + kS) + wave * kWave, (int)(sat + past), from * 4);
    };
    // the lane's units of any row it reads: 2 u + half, where the rotation has put them
    const int unit0 = rotate(r32, half);
    auto scales_of = [&](const u32x4 *from, int i, float (&scale)[2]) {
        const float *s = reinterpret_cast<const float *>(from + kS);
        const int r = wm * 32 * MI + i * 32 + r32;
        scale[0] = s[r] * s[BM + (SWIGLU ? 0 : wn >> 1)];
        scale[1] = SWIGLU ? s[r] * s[BM + 1] : scale[0];
    };
    auto add = [&](f32x16 &sum, const f32x16 &part, float scale) {
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e] = __builtin_fmaf(part[e], scale, sum[e]);
    };
    load(s_0, 0);
    load(s_1, 1);
    end_step<kLoads>();
    auto multiply = [&](const u32x4 *from) {
        const u32x4 *x = from + kX, *w = from + kW;
        int u0 = unit0;
        asm volatile("" : "+v"(u0));  // addresses are cheaper formed anew than kept in registers
        auto unit_of = [&](const u32x4 *rows, int r, int u) { return rows[r * kUnits + (u0 ^ (2 * u))]; };
        f16x8 fw[2][8];  // the wave's weights
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const u32x4 unit = unit_of(w, wn * 64 + j * 32 + r32, u);
                fw[j][2 * u] = to_f16<0>(unit);
                fw[j][2 * u + 1] = to_f16<1>(unit);
            }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            f32x16 part[2] = {};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const u32x4 unit = unit_of(x, wm * 32 * MI + i * 32 + r32, u);
                const f16x8 a = to_f16<0>(unit), b = to_f16<1>(unit);
                part[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fw[0][2 * u], a, part[0], 0, 0, 0);
                part[1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fw[1][2 * u], a, part[1], 0, 0, 0);
                part[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fw[0][2 * u + 1], b, part[0], 0, 0, 0);
                part[1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fw[1][2 * u + 1], b, part[1], 0, 0, 0);
            }
            float scale[2];
            scales_of(from, i, scale);
            add(acc[i][0], part[0], scale[0]);
            add(acc[i][1], part[1], scale[1]);
        }
    };
    // one block of channels: start the loads of the second next, multiply, let the next one's land
    auto step = [&](const u32x4 *now, u32x4 *later, int b) {
        load(later, b + 2);
        if (busy) multiply(now);
        end_step<kLoads>();
    };
    // (three steps a turn and no way round any of them: else the compiler would find loads under way
    // that no path has there, and wait for them)
    int b = 0;
    for (; b + 3 <= blocks; b += 3) {
        step(s_0, s_2, b);
        step(s_1, s_0, b + 1);
        step(s_2, s_1, b + 2);
    }
    if (b < blocks) step(s_0, s_2, b);
    if (b + 1 < blocks) step(s_1, s_0, b + 1);

    // The lane's element e of a 32 x 32 result: row r32, weight row 8 (e / 4) + 4 half + e % 4.  A
    // direct store would put 16 bytes into each of 32 rows; results go through LDS instead and out as
    // whole rows (32768 rows x 7168, 2048 channels: 731 -> 675 us, and 657 past the caches).
    end_step<0>();  // nothing reads the buffers or writes to them any more
    if constexpr (!SWIGLU) {
        // the rows of each half of the block in a buffer of their own, 512 bytes a row, 16-byte units
        // rotated by the row
        static_assert(32 * MI * kBN * 2 <= kBuffer * 16, "half the block's rows fit a buffer");
        u32x4 *rows = wm == 0 ? s_0 : s_1;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = i * 32 + r32;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint2 o;
                    o.x = pack_bf16(acc[i][j][4 * g], acc[i][j][4 * g + 1]);
                    o.y = pack_bf16(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
                    reinterpret_cast<uint2 *>(rows + r * 32 + ((wn * 8 + j * 4 + g) ^ r32))[half] = o;
                }
            }
        }
        __syncthreads();
        uint16_t *out = static_cast<uint16_t *>(p.out);
        const int unit = lane & 31, c = col_tile * kBN + unit * 8;
        for (int r = wn * 2 + (lane >> 5); r < 32 * MI; r += 2 * WN) {
            const int row = wm * 32 * MI + r;
            if (row >= t.rows || c >= p.n) continue;  // n is a multiple of 8: all eight or none
            __builtin_nontemporal_store(rows[r * 32 + (unit ^ (r & 31))],
                                        reinterpret_cast<u32x4 *>(out + (t.first + row) * p.n + c));
        }
    } else {
        float *s_top = reinterpret_cast<float *>(s_0);  // [WN][BM]: the tiles are done with
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float g = acc[i][0][e], u = acc[i][1][e];
                const float a = g / (1.0f + expf(-g)) * u;
                acc[i][0][e] = a;
                top = fmaxf(top, fabsf(a));
            }
            top = fmaxf(top, __shfl_xor(top, 32));
            if (half == 0) s_top[wn * BM + wm * 32 * MI + i * 32 + r32] = top;
        }
        __syncthreads();
        uint32_t *codes = reinterpret_cast<uint32_t *>(s_1);  // [BM][32] words, 16-byte units rotated by the row
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = wm * 32 * MI + i * 32 + r32;
            float m = kE4m3AmaxFloor;
#pragma unroll
            for (int j = 0; j < WN; ++j) m = fmaxf(m, s_top[j * BM + r]);
            const float inv = kE4m3Max / m;
            if (wn == 0 && half == 0 && r < t.rows)
                p.out_scales[(t.first + r) * (p.n / kScaleBlock) + col_tile] = m / kE4m3Max;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int word = wn * 8 + g * 2 + half;
                codes[r * 32 + ((word >> 2) ^ (r & 7)) * 4 + (word & 3)] =
                    e4m3_pack4(acc[i][0][4 * g] * inv, acc[i][0][4 * g + 1] * inv, acc[i][0][4 * g + 2] * inv,
                               acc[i][0][4 * g + 3] * inv);
            }
        }
        __syncthreads();
        uint8_t *out = static_cast<uint8_t *>(p.out);
        for (int i = threadIdx.x; i < BM * kUnits; i += kBlockThreads) {
            const int r = i / kUnits, unit = i % kUnits;
            if (r >= t.rows) continue;
            *reinterpret_cast<u32x4 *>(out + (t.first + r) * p.n + col_tile * 128 + unit * 16) =
                s_1[r * kUnits + (unit ^ (r & 7))];
        }
    }
}

// Few rows: 16 MF rows x 16 WF NG weight rows a block of NG x KS waves, WAVES of them a SIMD.  Each wave
// reads weights of its own, once, into registers, DEEP blocks of channels at a time, and there are no
// barriers: a wave has loads under way while it multiplies.  The KS waves of a group take every KS-th
// block of channels and add up through LDS at the end.
//
// With rows for many experts this is bound by the weights' bytes: 128 rows of 32 experts take 162 us
// for 0.94 GB (SwiGLU, 7168 channels to 2048) and 77 us for 0.47 GB (product, 2048 to 7168), 5.8 and
// 6.1 TB/s.  A few blocks alone are bound by what one compute unit takes in: 16 bytes a clock where
// neighbouring lanes read different rows, as the matrix instructions want them, and over 30 where eight
// lanes read a row's 128 bytes.  So they do that, and the wave turns its tile round in LDS that no other
// wave touches (16 rows of one expert, 2048 of 7168 channels: 23 -> 12 us; the SwiGLU above 180 -> 162).
template <bool SWIGLU, int MF, int WF, int NG, int KS, int DEEP, int WAVES>
__global__ __launch_bounds__(NG *KS *kWave, WAVES) void expert_gemm_narrow_kernel(GemmArgs p, int col_tiles) {
    static_assert(!SWIGLU || 8 * WF * NG == 128, "a block holds a scale's 128 outputs");
    constexpr int BM = 16 * MF, BN = 16 * WF * NG;
    constexpr int SETS = SWIGLU ? WF / 2 : WF;  // 16 columns of output each, of a group
    constexpr int XL = 2 * MF, WL = 2 * WF;     // loads of a block's rows and weight rows, 8 rows each
    constexpr int kTile = (XL + WL) * kWave;
    constexpr int kSums = WF * MF * kWave;
    constexpr int kShare = kTile > kSums ? kTile : kSums;  // of a wave: its tile, then its sums
    __shared__ u32x4 s_tile[NG * KS][kShare];
    __shared__ float s_top[NG][SETS][BM];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave % NG, ks = wave / NG;
    const int col_tile = blockIdx.x % col_tiles;
    const Tile t = find_tile(p, BM, blockIdx.x / col_tiles, blockIdx.x == 0);
    if (t.rows == 0) return;  // the whole block: every wave found the same
    const int wrows = SWIGLU ? 2 * p.n : p.n;
    const int blocks = p.k / kScaleBlock;
    const int scale_rows = (wrows + kScaleBlock - 1) / kScaleBlock;
    const __amdgpu_buffer_rsrc_t xbuf = descriptor(p.x + t.first * p.k, (uint32_t)t.rows * p.k);
    const __amdgpu_buffer_rsrc_t wbuf = descriptor(p.w + (int64_t)t.expert * wrows * p.k, (uint32_t)wrows * p.k);
    const __amdgpu_buffer_rsrc_t sbuf = descriptor(p.x_scales + t.first * blocks, (uint32_t)t.rows * blocks * 4);

    // rows past the segment and weight rows past the last are past the descriptors' ends: they read
    // as 0 and are not stored
    const int q = lane >> 4, r16 = lane & 15;
    const uint32_t k = p.k;  // unsigned: a row past the end may lie past 2^31, and must not come out below 0
    const int sat = r16 * blocks * 4;
    // column (output) of the group's first weight row; SWIGLU: half are gate rows, half the up rows of the same
    const int c0 = SWIGLU ? col_tile * 128 + group * 8 * WF : col_tile * BN + group * 16 * WF;
    // eight lanes load a row's 128 bytes, unit c of row r to place c ^ (r / 2) % 8 of its row in LDS
    const int r8 = lane >> 3;
    const uint32_t unit[2] = {(uint32_t)((lane & 7) ^ (r8 >> 1)) * 16, (uint32_t)((lane & 7) ^ (r8 >> 1) ^ 4) * 16};
    const uint32_t xat = r8 * k, wat = (uint32_t)(c0 + r8) * k;
    const float *sw0 = p.w_scales + (int64_t)t.expert * scale_rows * blocks;
    const float *sw1;
    if constexpr (SWIGLU) {
        sw1 = sw0 + (int64_t)(p.n / kScaleBlock + col_tile) * blocks;
        sw0 += (int64_t)col_tile * blocks;
    } else {
        sw0 += (int64_t)(c0 / kScaleBlock < scale_rows ? c0 / kScaleBlock : scale_rows - 1) * blocks;
        sw1 = sw0;
    }

    struct Codes {
        u32x4 w[WL], x[XL];
        float sx[MF], sw[2];
    };
    // Past the last block the loads go on, from behind the descriptors' ends (they fetch nothing):
    // that every step issues the same number is what lets the waits count.
    auto load = [&](Codes &c, int b) {
        const uint32_t past = b < blocks ? 0u : 0x80000000u;
        const int from = b < blocks ? b : 0;
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const uint32_t row = SWIGLU && i >= WL / 2 ? p.n + (i - WL / 2) * 8 : i * 8;
            c.w[i] = __builtin_amdgcn_raw_buffer_load_b128(wbuf, (int)(wat + row * k + unit[i & 1] + past), from * kScaleBlock, 0);
        }
#pragma unroll
        for (int i = 0; i < XL; ++i)
            c.x[i] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, (int)(xat + i * 8 * k + unit[i & 1] + past), from * kScaleBlock, 0);
#pragma unroll
        for (int i = 0; i < MF; ++i)
            c.sx[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sbuf, sat + i * 16 * blocks * 4, from * 4, 0));
        c.sw[0] = sw0[from];
        c.sw[1] = SWIGLU ? sw1[from] : c.sw[0];
    };
    u32x4 *tile = s_tile[wave];
    const int place = q ^ (r16 >> 1);
    auto unit_of = [&](int row, int h) { return tile[(row + r16) * kUnits + (place ^ (4 * h))]; };
    f32x4 acc[MF][WF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < WF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Codes &c) {
#pragma unroll
        for (int i = 0; i < WL; ++i) tile[i * kWave + lane] = c.w[i];
#pragma unroll
        for (int i = 0; i < XL; ++i) tile[(WL + i) * kWave + lane] = c.x[i];
        wave_lds_order();
        u32x4 x[MF][2];
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            x[i][0] = unit_of(16 * (WF + i), 0);
            x[i][1] = unit_of(16 * (WF + i), 1);
        }
#pragma unroll
        for (int j = 0; j < WF; ++j) {
            f16x8 fw[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 w = unit_of(j * 16, h);
                fw[2 * h] = to_f16<0>(w);
                fw[2 * h + 1] = to_f16<1>(w);
            }
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(fw[2 * h], to_f16<0>(x[i][h]), part, 0, 0, 0);
                    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(fw[2 * h + 1], to_f16<1>(x[i][h]), part, 0, 0, 0);
                }
                const float s = c.sx[i] * c.sw[SWIGLU && j >= SETS];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[e], s, acc[i][j][e]);
            }
        }
        wave_lds_order();  // the next tile, or the sums, go where this one was
    };
    Codes c[DEEP];
#pragma unroll
    for (int d = 0; d + 1 < DEEP; ++d) load(c[d], ks + d * KS);
    for (int b = ks; b < blocks; b += DEEP * KS) {
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            load(c[(d + DEEP - 1) % DEEP], b + (d + DEEP - 1) * KS);
            if (b + d * KS < blocks) multiply(c[d]);
        }
    }

    // the KS sums of each 16 x 16 result, added in order; the waves of a group share its results out
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < WF; ++j) reinterpret_cast<f32x4 *>(tile)[(j * MF + i) * kWave + lane] = acc[i][j];
    __syncthreads();
    auto total = [&](int j, int i) {
        auto part = [&](int k) {
            return reinterpret_cast<const f32x4 *>(s_tile[k * NG + group])[(j * MF + i) * kWave + lane];
        };
        f32x4 v = part(0);
#pragma unroll
        for (int k = 1; k < KS; ++k) v += part(k);
        return v;
    };
    constexpr int SHARE = (SETS * MF + KS - 1) / KS;  // results a wave finishes, at most
    if constexpr (!SWIGLU) {
        uint16_t *out = static_cast<uint16_t *>(p.out);
#pragma unroll
        for (int o = 0; o < SHARE; ++o) {
            const int u = o * KS + ks, j = u % SETS, i = u / SETS;
            if (u >= SETS * MF) break;
            const f32x4 v = total(j, i);
            const int r = i * 16 + r16, c = c0 + j * 16 + q * 4;
            if (r >= t.rows || c >= p.n) continue;  // n is a multiple of 8: all four or none
            uint2 pair;
            pair.x = pack_bf16(v[0], v[1]);
            pair.y = pack_bf16(v[2], v[3]);
            *reinterpret_cast<uint2 *>(out + (t.first + r) * p.n + c) = pair;
        }
    } else {
        f32x4 a[SHARE];
#pragma unroll
        for (int o = 0; o < SHARE; ++o) {
            const int u = o * KS + ks, j = u % SETS, i = u / SETS;
            if (u >= SETS * MF) break;
            const f32x4 g = total(j, i), v = total(SETS + j, i);
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[o][k] = g[k] / (1.0f + expf(-g[k])) * v[k];
                top = fmaxf(top, fabsf(a[o][k]));
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            if (q == 0) s_top[group][j][i * 16 + r16] = top;
        }
        __syncthreads();
        uint8_t *out = static_cast<uint8_t *>(p.out);
#pragma unroll
        for (int o = 0; o < SHARE; ++o) {
            const int u = o * KS + ks, j = u % SETS, i = u / SETS;
            if (u >= SETS * MF) break;
            const int r = i * 16 + r16;
            if (r >= t.rows) continue;
            float m = kE4m3AmaxFloor;
#pragma unroll
            for (int n = 0; n < NG * SETS; ++n) m = fmaxf(m, s_top[n / SETS][n % SETS][r]);
            const float inv = kE4m3Max / m;
            if (group == 0 && j == 0 && q == 0)
                p.out_scales[(t.first + r) * (p.n / kScaleBlock) + col_tile] = m / kE4m3Max;
            *reinterpret_cast<uint32_t *>(out + (t.first + r) * p.n + c0 + j * 16 + q * 4) =
                e4m3_pack4(a[o][0] * inv, a[o][1] * inv, a[o][2] * inv, a[o][3] * inv);
        }
    }
}

int64_t row_tiles(const GemmArgs &a, int bm) {
    if (a.expert_rows == nullptr) return ((int64_t)a.num_rows + bm - 1) / bm;
    const int64_t busy = a.num_experts < a.num_rows ? a.num_experts : a.num_rows;
    return a.num_rows / bm + busy;  // each segment ends in at most one part tile
}

// A kernel for a product, and what a block of it works on.
struct Plan {
    void (*kernel)(GemmArgs, int);
    int threads, rows, cols;
};

template <bool SWIGLU, int MF, int WF, int NG, int KS, int DEEP, int WAVES>
Plan narrow() {
    return {expert_gemm_narrow_kernel<SWIGLU, MF, WF, NG, KS, DEEP, WAVES>, NG * KS * kWave, 16 * MF,
            SWIGLU ? 128 : 16 * WF * NG};
}

// The choice rests on the mean rows of an expert, all that the host knows of the sizes.  Measured
// over 32 experts, SwiGLU of 7168 channels to 2048 and product of 2048 to 7168, us (s: narrow<...> by
// its MF, WF, NG and KS):
//   mean rows               4    8   12   16   24   32   48   64   96  128  192  256  512
//   SwiGLU   s 1, 4, 4, 2 165  165  194  192  237  262
//            s 2, 4, 4, 2 170  168  170  172  217  229
//            wide 64      163  163  163  164  165  168  175  237  297  388  532  664 1181
//            wide 128     168  168  168  169  169  173  173  219  248  388  477  601 1051
//   product  s 1, 4, 1, 8  81   83   87   97  119  135  174  215
//            s 2, 4, 1, 8 112  116  116  117  126  152  196  237
//            s 2, 4, 2, 2  86   89   88   90   97  109  127  148  194
//            wide 64       96   94   99   99   99  101  107  124  157  200  283  345  636
//            wide 128     104  104  105  105  106  107  107  137  143  181  247  297  549
// Where there are fewer blocks than compute units a block's own time counts, and more waves of a block
// on the channels, or fewer columns a block, shorten it.  One expert, product of 7168 channels to 2048
// and of 2048 to 7168, and SwiGLU of 7168 to 2048, us:
//   rows                    1   16   64  128  256  512 1024 2048 4096 |   1   64  128  256  512 1024 2048 4096
//   product  s 1, 1, 1, 8   7    8   14   25   46                     |   6   20   37
//            s 1, 4, 1, 8  11   12   12   14   23   39   76           |   6   10   16   25   46
//            s 2, 4, 1, 8  15   15   17   17   18   33   64  121      |   8    8   15   27   47   89
//            s 2, 4, 2, 2  33   32   34   34   35   38   56  102  186 |  12   13   14   21   34   57  106
//            wide 64       36   37   58   58   59   61   63   80  151 |  13   20   20   21   23   43   87  158
//            wide 128      52   53   54   86   87   88   89   94  126 |  18   19   29   30   31   34   74  136
//   SwiGLU   s 1, 4, 4, 2  36   37   37   37   40   79  151
//            s 2, 4, 4, 2  43   44   47   46   47   52  101  199
//            wide 64       38   39   59   60   61   64   81  151  285
//            wide 128      57   57   57   90   91   93   96  133  236
constexpr int kComputeUnits = 256;
Plan plan(const GemmArgs &a) {
    const int64_t mean = a.num_rows / a.num_experts;
    const int64_t busy = a.num_experts < a.num_rows ? a.num_experts : a.num_rows;
    // blocks to expect: a segment's last tile is half full on average
    auto blocks = [&](int rows, int cols) {
        int64_t tiles = (a.num_rows + busy * rows / 2) / rows;
        if (a.num_experts == 1) tiles = ((int64_t)a.num_rows + rows - 1) / rows;
        return (tiles > busy ? tiles : busy) * ((a.n + cols - 1) / cols);
    };
    if (a.swiglu) {
        if (mean <= 8 || blocks(16, 128) <= kComputeUnits) return narrow<true, 1, 4, 4, 2, 2, 2>();
        if (blocks(32, 128) <= kComputeUnits) return narrow<true, 2, 4, 4, 2, 2, 2>();
        if (mean <= 32 || blocks(64, 128) <= kComputeUnits)
            return {expert_gemm_wide_kernel<true, 1>, kBlockThreads, 64, 128};
        return {expert_gemm_wide_kernel<true, 2>, kBlockThreads, 128, 128};
    }
    if (blocks(16, 16) <= kComputeUnits) return narrow<false, 1, 1, 1, 8, 3, 2>();
    if (mean <= 12 || blocks(16, 64) <= kComputeUnits) return narrow<false, 1, 4, 1, 8, 2, 2>();
    if (blocks(32, 64) <= 2 * kComputeUnits) return narrow<false, 2, 4, 1, 8, 2, 2>();
    if (mean <= 24 || blocks(32, 128) <= 2 * kComputeUnits) return narrow<false, 2, 4, 2, 2, 2, 3>();
    // rounds of blocks over the compute units, whole rounds where there are few; a round of 128 rows
    // takes 1.5 times one of 64
    auto time = [&](int rows) {
        const int64_t all = blocks(rows, kBN), rounds = (all + kComputeUnits - 1) / kComputeUnits;
        return rounds <= 2 ? rounds * kComputeUnits : all;
    };
    if (2 * time(64) <= 3 * time(128)) return {expert_gemm_wide_kernel<false, 1>, kBlockThreads, 64, kBN};
    return {expert_gemm_wide_kernel<false, 2>, kBlockThreads, 128, kBN};
}

int64_t grid_blocks(const GemmArgs &a, const Plan &pl) {
    return row_tiles(a, pl.rows) * ((a.n + pl.cols - 1) / pl.cols);
}

}  // namespace

bool gemm_grid_ok(const GemmArgs &a) {
    const Plan pl = plan(a);
    return grid_blocks(a, pl) <= INT_MAX / pl.threads;
}

hipError_t launch_expert_gemm(const GemmArgs &a, hipStream_t stream) {
    const Plan pl = plan(a);
    int64_t blocks = grid_blocks(a, pl);
    if (blocks == 0) {  // no rows: nothing but sizes that say there are some
        if (a.expert_rows == nullptr || a.dev_status == nullptr) return hipSuccess;
        blocks = 1;
    }
    return start_kernel(pl.kernel, blocks, pl.threads, stream, a, (a.n + pl.cols - 1) / pl.cols);
}

}  // namespace ep

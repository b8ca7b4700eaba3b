// decode_tile.cuh -- the tensor-core key tile that the decode kernels share (decode.cu,
// decode_shared.cu).
#pragma once

#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

constexpr int kTileKeys = 64;
constexpr int kD = 128;
constexpr int kMaxRows = 32;                    // G * T

// Per-warp attention state for one m-tile of 16 query rows.
struct RowState {
    float o[kD / 8][4];
    float m[2];
    float l[2];
};

// Running max may lag the true one by up to this much (log2 units) before O is
// rescaled: P then stays below 2^8, exact enough in bf16, and most tiles skip the
// 64-register rescale of O.
constexpr float kRescaleSlack = 8.0f;

// m16n8k16 MMA and operand packing in bf16, or fp16 when F16 is set.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    if (F16)
        mma_f16_16816(d, a, b0, b1);
    else
        mma_bf16_16816(d, a, b0, b1);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    return F16 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
}

// One key tile on tensor cores.  NT = n-tiles of 8 keys this warp owns inside the
// tile (keys key0 .. key0 + 8 NT - 1), rows = the tile's row count in shared
// memory (for the swizzle), vis(row, key) = key visible to that query row; when
// all_vis is set every key of the tile is visible to every valid row and only rows
// past G T (padding) are masked.
// F16: the operands (Q fragments and the tile in shared memory) are fp16 instead
// of bf16 (the FP8 kernel's new-token tile).
template <int NT, bool F16 = false, typename Vis>
__device__ __forceinline__ void run_tile(RowState &st, const uint32_t (&qa)[kD / 16][4],
                                         uint32_t sK, uint32_t sV, int tile_rows, int key0,
                                         float scale_log2, bool all_vis, bool row0_ok,
                                         bool row1_ok, Vis vis)
{
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, tq = lane & 3;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;

    // S = Q K^T: B fragments via ldmatrix (rows = keys, cols = dims)
    {
        const int mi = lane >> 3, r = lane & 7;
#pragma unroll
        for (int np = 0; np < NT / 2; ++np) {
            const int key = key0 + np * 16 + (mi >> 1) * 8 + r;
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                const int dim = ks * 16 + (mi & 1) * 8;
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4(sK + swz128_offset(key, dim, tile_rows), b0, b1, b2, b3);
                mma16816<F16>(s[2 * np], qa[ks], b0, b1);
                mma16816<F16>(s[2 * np + 1], qa[ks], b2, b3);
            }
        }
    }

    // mask (raw scores; the scale is positive and folded into the exponent below)
    if (!all_vis) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int key = key0 + nt * 8 + 2 * tq + e;
                if (!vis(g, key))
                    s[nt][e] = -INFINITY;
                if (!vis(g + 8, key))
                    s[nt][2 + e] = -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (!row0_ok)
                s[nt][0] = s[nt][1] = -INFINITY;
            if (!row1_ok)
                s[nt][2] = s[nt][3] = -INFINITY;
        }
    }
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        mx0 = fmaxf(mx0, fmaxf(s[nt][0], s[nt][1]));
        mx1 = fmaxf(mx1, fmaxf(s[nt][2], s[nt][3]));
    }
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    mx0 *= scale_log2;
    mx1 *= scale_log2;
    // running max, raised lazily (the quad shares a row, so its decision is uniform)
    const bool up0 = mx0 != -INFINITY && (st.m[0] == -INFINITY || mx0 > st.m[0] + kRescaleSlack);
    const bool up1 = mx1 != -INFINITY && (st.m[1] == -INFINITY || mx1 > st.m[1] + kRescaleSlack);
    if (__any_sync(0xffffffffu, up0 || up1)) {
        const float a0 = up0 ? fast_exp2(st.m[0] - mx0) : 1.f;  // m = -inf: O is still 0
        const float a1 = up1 ? fast_exp2(st.m[1] - mx1) : 1.f;
        if (up0)
            st.m[0] = mx0;
        if (up1)
            st.m[1] = mx1;
        st.l[0] *= a0;
        st.l[1] *= a1;
#pragma unroll
        for (int n = 0; n < kD / 8; ++n) {
            st.o[n][0] *= a0;
            st.o[n][1] *= a0;
            st.o[n][2] *= a1;
            st.o[n][3] *= a1;
        }
    }
    const float base0 = st.m[0] == -INFINITY ? 0.f : st.m[0];
    const float base1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        s[nt][0] = fast_exp2(fmaf(s[nt][0], scale_log2, -base0));
        s[nt][1] = fast_exp2(fmaf(s[nt][1], scale_log2, -base0));
        s[nt][2] = fast_exp2(fmaf(s[nt][2], scale_log2, -base1));
        s[nt][3] = fast_exp2(fmaf(s[nt][3], scale_log2, -base1));
    }

    // O += P V: P from the S accumulators, V fragments via ldmatrix.trans.  The row
    // sums take the same bf16-rounded P the MMA uses, so O / l is an exact convex
    // combination of V rows (no scale error proportional to |O|).
    const int mi = lane >> 3, r = lane & 7;
    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
    for (int ks = 0; ks < NT / 2; ++ks) {
        uint32_t pa[4];
        pa[0] = pack16<F16>(s[2 * ks][0], s[2 * ks][1]);
        pa[1] = pack16<F16>(s[2 * ks][2], s[2 * ks][3]);
        pa[2] = pack16<F16>(s[2 * ks + 1][0], s[2 * ks + 1][1]);
        pa[3] = pack16<F16>(s[2 * ks + 1][2], s[2 * ks + 1][3]);
        if constexpr (F16) {
            sum0 += f16_lo(pa[0]) + f16_hi(pa[0]) + f16_lo(pa[2]) + f16_hi(pa[2]);
            sum1 += f16_lo(pa[1]) + f16_hi(pa[1]) + f16_lo(pa[3]) + f16_hi(pa[3]);
        } else {
            sum0 += bf16_lo(pa[0]) + bf16_hi(pa[0]) + bf16_lo(pa[2]) + bf16_hi(pa[2]);
            sum1 += bf16_lo(pa[1]) + bf16_hi(pa[1]) + bf16_lo(pa[3]) + bf16_hi(pa[3]);
        }
        const int key = key0 + ks * 16 + (mi & 1) * 8 + r;
#pragma unroll
        for (int np = 0; np < kD / 16; ++np) {
            const int dim = np * 16 + (mi >> 1) * 8;
            uint32_t b0, b1, b2, b3;
            ldmatrix_x4_trans(sV + swz128_offset(key, dim, tile_rows), b0, b1, b2, b3);
            mma16816<F16>(st.o[2 * np], pa, b0, b1);
            mma16816<F16>(st.o[2 * np + 1], pa, b2, b3);
        }
    }
    st.l[0] += sum0;
    st.l[1] += sum1;
}

}  // namespace
}  // namespace hsa

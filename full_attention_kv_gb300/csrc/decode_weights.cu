// decode_weights.cu -- decode attention over a full layer that also weighs its keys (sm_103a).
//
// What it computes: for sequence b, KV head h and query row (t, hh) at position c + t,
//   s_j = scale q.k_j (j <= c + t),  lse = log sum exp s_j,  o = sum exp(s_j - lse) v_j,
//   w_j = decay w_prev_j + sum over the G T rows of exp(s_j - lse).
// A weight needs its row's lse, which is known once every key has been seen, while the keys are
// worth reading only once (512 bytes a key and head in bf16).  So the scores are kept: 4 G T
// bytes a key, written beside the attention and read again when the states are joined.
//
// attend_kernel: the 64-key pages of all (sequence, KV head) units are laid end to end and cut
// into equal contiguous ranges, one a CTA (one CTA an SM).  A producer warp streams pages by TMA
// into a ring of stages; the consumer warps take whole pages in turn (groups of RH warps, each 8
// NT of the unit's rows), operands swapped: S^T = K Q^T has the keys on the MMA's M side and the
// rows on its N side, so 8 rows waste nothing, a thread holds two rows of a key side by side, and
// the scores leave in 256-byte runs a warp.  O^T += V^T P^T, P through 8x8 transposes.  Every
// group keeps a state of its own from a unit's first page in the range to its last and writes it
// to the workspace: no barrier among the consumers.  The new tokens are a tile of 16 keys that
// one group takes at the unit's end.
//
// join_kernel: chunks of positions of all units, cut evenly.  A unit's states (those of the
// CTAs whose ranges met it lie side by side) give lse; then two floats to four a thread, the
// scores become weights and are summed over the rows by shuffles.  Eight rows of output are an
// item of their own.  The order of every sum is fixed by the sizes.
//
// What bounds it: HBM, the reads of K and V and the scores' way out and in.  Attend and, behind it,
// join: 32 sequences of 8192 to 65536 tokens, 8 rows a head: 424 us (6.4 TB/s of K and V, 0.94 of a
// copy's rate, scores beside them) and 41.  32 rows a head (16 sequences of 3001 to 20000 x 4 tokens):
// 83 and 27; about 10 us of it are the kernel's start and end, in the join instructions (issue 50%).
// FP8, 8 sequences of 8192 to 65536: 50 and 20, the same; 32 rows a head as above: 92 and 22, one warp
// a scheduler, bound by its chain a page.  (Six consuming warps and stages, FP8 six to twelve: no
// change.)
#include "decode_tile.cuh"
#include "fp8_kv.cuh"
#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

constexpr int kNewKeys = 16;                     // new-token tile (T <= 4 used)
constexpr int kTileBytes = kTileKeys * kD * 2;   // one K or V tile, bf16
constexpr int kFp8TileBytes = kTileKeys * kD;
constexpr int kFp8StageStride = 17408;           // codes of K and V, 2 x 64 scales, up to 1 KB
constexpr int kLens = 1024;                      // sequences whose lengths are kept on chip
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 3;                     // of it, an SM (85 registers a thread)
constexpr int kBatch = 6;                        // loads of scores a thread has on the way (4, 8: no better)
constexpr float kUnused = -1.f;                  // sum of the rounded weights of a group without keys

// Warps, groups and stages of an instantiation.  A stage belongs to one group (the stages are a
// multiple of the groups), so that a parity never stands for two of its phases.
template <int FP8, int NT, int RH>
struct Shape {
    static constexpr int kWarps = FP8 && NT == 1 ? 8 : 4;
    static constexpr int kGroups = kWarps / RH;
    static constexpr int kStages = FP8 ? 8 : 4;
    static constexpr int kStageStride = FP8 ? kFp8StageStride : 2 * kTileBytes;
    static constexpr int kThreads = (kWarps + 1) * 32;
    static_assert(kStages % kGroups == 0, "each stage belongs to one group");
};

template <int FP8, int NT, int RH>
struct alignas(1024) AttendSmem {
    using S = Shape<FP8, NT, RH>;
    uint8_t stage[S::kStages * S::kStageStride];
    alignas(1024) uint8_t new_k[RH][kNewKeys * kD * 2];
    alignas(1024) uint8_t new_v[RH][kNewKeys * kD * 2];
    alignas(8) uint64_t full[8], empty[8];
    int32_t tile_ok[8];
    int32_t len[kLens];
    int32_t scan[S::kThreads];
    int32_t first_b, before, total;
};

// Cached tokens of sequence b, or -1 if it is left out.
__device__ __forceinline__ int seq_len(const WeighParams &p, int b)
{
    const int c = max(0, __ldg(p.cached_len + b));
    return c > p.w_stride - p.T ? -1 : c;
}

__device__ __forceinline__ int pages_of(int c)
{
    return c < 0 ? 0 : max(1, (int)(((int64_t)c + kTileKeys - 1) / kTileKeys));
}

// Exclusive scan of one value a thread over the block (kThr threads, a multiple of 32);
// shared[kThr] holds the result, the total comes back.  Two barriers.
template <int kThr>
__device__ __forceinline__ int block_scan(int32_t *shared, int32_t *total, int value, int tid)
{
    constexpr int kPer = kThr / 32;
    shared[tid] = value;
    __syncthreads();
    if (tid < 32) {
        int v[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            v[j] = shared[tid * kPer + j];
            sum += v[j];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (tid >= o)
                incl += u;
        }
        int acc = incl - sum;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            shared[tid * kPer + j] = acc;
            acc += v[j];
        }
        if (tid == 31)
            *total = incl;
    }
    __syncthreads();
    return *total;
}

struct UnitWalk {
    int b, h, j, n, c;  // sequence, head, page j of n, cached tokens
};

// A state's place in the workspace: m[RP], l[RP], the sum of the rounded weights[RP], o[RP][d].
__host__ __device__ constexpr int slot_floats(int rows_padded) { return rows_padded * (kD + 3); }

template <int NT>
struct State {
    float m[NT][2], l[NT][2], lr[NT][2];  // lr: of the weights as the product takes them
    float o[kD / 16][NT][4];
};

template <int NT>
__device__ __forceinline__ void clear(State<NT> &st)
{
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st.m[n][e] = -INFINITY;
            st.l[n][e] = st.lr[n][e] = 0.f;
        }
#pragma unroll
    for (int dt = 0; dt < kD / 16; ++dt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                st.o[dt][n][e] = 0.f;
}

// The running maxima raised by a tile's (x, in log2 units, the same in all lanes of a column);
// lazily, as in run_tile.
template <int NT>
__device__ __forceinline__ void raise(State<NT> &st, const float (&x)[NT][2])
{
    bool up[NT][2], any = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            up[n][e] = x[n][e] != -INFINITY &&
                       (st.m[n][e] == -INFINITY || x[n][e] > st.m[n][e] + kRescaleSlack);
            any |= up[n][e];
        }
    if (!__any_sync(0xffffffffu, any))
        return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            a[e] = up[n][e] ? fast_exp2(st.m[n][e] - x[n][e]) : 1.f;
            if (up[n][e])
                st.m[n][e] = x[n][e];
            st.l[n][e] *= a[e];
            st.lr[n][e] *= a[e];
        }
#pragma unroll
        for (int dt = 0; dt < kD / 16; ++dt) {
            st.o[dt][n][0] *= a[0];
            st.o[dt][n][1] *= a[1];
            st.o[dt][n][2] *= a[0];
            st.o[dt][n][3] *= a[1];
        }
    }
}

// Column maxima of a tile's scaled scores over the warp's keys.
template <int NT, int MTS>
__device__ __forceinline__ void column_max(const float (&s)[MTS][NT][4], float (&x)[NT][2])
{
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float y = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MTS; ++mt)
                y = fmax3(y, s[mt][n][e], s[mt][n][2 + e]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
            x[n][e] = y;
        }
    }
}

// A tile's scores to the workspace: key k of the tile is score row `to + k srow`, this warp's
// columns from col0; keys >= valid are not stored.
template <int NT, int MTS>
__device__ __forceinline__ void store_scores(const float (&s)[MTS][NT][4], float *to, int srow, int col0,
                                             int valid, int lane)
{
    const int g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int col = col0 + n * 8 + 2 * tq;
        if (col >= srow)
            continue;
#pragma unroll
        for (int mt = 0; mt < MTS; ++mt) {
            const int a = mt * 16 + g;
            if (a < valid)
                *reinterpret_cast<float2 *>(to + (int64_t)a * srow + col) =
                    make_float2(s[mt][n][0], s[mt][n][1]);
            if (a + 8 < valid)
                *reinterpret_cast<float2 *>(to + (int64_t)(a + 8) * srow + col) =
                    make_float2(s[mt][n][2], s[mt][n][3]);
        }
    }
}

// A bf16 tile of 16 MTS keys in shared memory (rows of the swizzle: tile_rows).  Keys >= valid
// and, of the new tokens (causal), those after a row's own are masked: row r sees key <= r / G.
// P rounds to bf16 for the product with V, 2^-9 of itself whatever its size; the output is divided
// by the sum of the rounded ones (lr), the weights' lse takes the sum in fp32 (l).
template <int NT, int MTS>
__device__ __forceinline__ void tile_bf16(State<NT> &st, const uint32_t (&qb)[NT][kD / 16][2],
                                          uint32_t sK, uint32_t sV, int tile_rows, int valid,
                                          bool causal, int G, int col0, float scale_log2, float *score,
                                          int srow, int lane)
{
    const int g = lane >> 2, tq = lane & 3, mi = lane >> 3, r8 = lane & 7;
    float s[MTS][NT][4];
#pragma unroll
    for (int mt = 0; mt < MTS; ++mt) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks) {
            uint32_t a[4];
            ldmatrix_x4(sK + swz128_offset(mt * 16 + (mi & 1) * 8 + r8, ks * 16 + (mi >> 1) * 8, tile_rows),
                        a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma_bf16_16816(s[mt][n], a, qb[n][ks][0], qb[n][ks][1]);
        }
    }
#pragma unroll
    for (int mt = 0; mt < MTS; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = mt * 16 + g + 8 * (e >> 1), row = col0 + n * 8 + 2 * tq + (e & 1);
                const bool seen = key < valid && !(causal && key * G > row);
                s[mt][n][e] = seen ? s[mt][n][e] * scale_log2 : -INFINITY;
            }
    store_scores<NT, MTS>(s, score, srow, col0, valid, lane);
    float x[NT][2];
    column_max<NT, MTS>(s, x);
    raise(st, x);
    float base[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            base[n][e] = st.m[n][e] == -INFINITY ? 0.f : st.m[n][e];
#pragma unroll
    for (int mt = 0; mt < MTS; ++mt) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float p0 = fast_exp2(s[mt][n][0] - base[n][0]), p1 = fast_exp2(s[mt][n][1] - base[n][1]);
            const float p2 = fast_exp2(s[mt][n][2] - base[n][0]), p3 = fast_exp2(s[mt][n][3] - base[n][1]);
            const uint32_t lo = pack_bf16(p0, p1), hi = pack_bf16(p2, p3);
            st.l[n][0] += p0 + p2;
            st.l[n][1] += p1 + p3;
            st.lr[n][0] += bf16_lo(lo) + bf16_lo(hi);
            st.lr[n][1] += bf16_hi(lo) + bf16_hi(hi);
            pb[n][0] = movmatrix_trans(lo);  // keys 0-7 of the 16
            pb[n][1] = movmatrix_trans(hi);  // keys 8-15
        }
#pragma unroll
        for (int dt = 0; dt < kD / 16; ++dt) {
            uint32_t a[4];
            ldmatrix_x4_trans(sV + swz128_offset(mt * 16 + (mi >> 1) * 8 + r8, dt * 16 + (mi & 1) * 8, tile_rows),
                              a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma_bf16_16816(st.o[dt][n], a, pb[n][0], pb[n][1]);
        }
    }
}

// A page of an FP8 layer (tile_fp8_sw in decode.cu says how its words feed the MMAs): fp16
// products, a key's scale on its scores, V's folded into P.  PART: keys >= valid are masked, their
// codes of V too.
//
// P times V's scale rounds to fp16, which is fine (2^-11 of itself, where bf16 has 2^-9) as long as
// it stays clear of fp16's small end.  So a row's are taken in units of a power of two that puts
// the page's largest between 2^14 and 2^15, and the page's product joins O in fp32, scaled back:
// those down to 2^-28 of a page's largest keep all their bits, those below are off by 2^-39 of it.
// A key of large V that has no weight, or of much weight that has no V, is no largest.
template <int NT, bool E5M2, bool PART>
__device__ __forceinline__ void tile_fp8(State<NT> &st, const uint32_t (&qb)[NT][kD / 16][2],
                                         const uint8_t *sK, const uint8_t *sV, const float *k_scale,
                                         const float *v_scale, int valid, int col0, float scale_log2,
                                         float *score, int srow, int lane)
{
    constexpr int MTS = kTileKeys / 16;
    const int g = lane >> 2, tq = lane & 3;
    float s[MTS][NT][4];
#pragma unroll
    for (int mt = 0; mt < MTS; ++mt) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
        const uint8_t *ra = sK + (mt * 16 + g) * 128 + 4 * tq, *rb = ra + 8 * 128;
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks) {
            const int off = (ks ^ g) << 4;
            const uint32_t wa = *reinterpret_cast<const uint32_t *>(ra + off);
            const uint32_t wb = *reinterpret_cast<const uint32_t *>(rb + off);
            const uint32_t a[4] = {fp8x2_lo<E5M2>(wa), fp8x2_lo<E5M2>(wb), fp8x2_hi<E5M2>(wa),
                                   fp8x2_hi<E5M2>(wb)};
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma_f16_16816(s[mt][n], a, qb[n][ks][0], qb[n][ks][1]);
        }
    }
#pragma unroll
    for (int mt = 0; mt < MTS; ++mt) {
        const int ka = mt * 16 + g, kb = ka + 8;
        const float sa = k_scale[ka] * scale_log2, sb = k_scale[kb] * scale_log2;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[mt][n][e] = PART && (e < 2 ? ka : kb) >= valid ? -INFINITY : s[mt][n][e] * (e < 2 ? sa : sb);
    }
    store_scores<NT, MTS>(s, score, srow, col0, PART ? valid : kTileKeys, lane);
    float x[NT][2];
    column_max<NT, MTS>(s, x);
    raise(st, x);
    // P V-scale in place of the scores, and each column's largest
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float base0 = st.m[n][0] == -INFINITY ? 0.f : st.m[n][0];
        const float base1 = st.m[n][1] == -INFINITY ? 0.f : st.m[n][1];
        top[n][0] = top[n][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < MTS; ++mt) {
            const int ka = mt * 16 + g, kb = ka + 8;
            const float va = !PART || ka < valid ? v_scale[ka] : 0.f;
            const float vb = !PART || kb < valid ? v_scale[kb] : 0.f;
            const float p0 = fast_exp2(s[mt][n][0] - base0), p1 = fast_exp2(s[mt][n][1] - base1);
            const float p2 = fast_exp2(s[mt][n][2] - base0), p3 = fast_exp2(s[mt][n][3] - base1);
            st.l[n][0] += p0 + p2;
            st.l[n][1] += p1 + p3;
            f2_split(f2_mul(f2_make(p0, p1), f2_make(va, va)), s[mt][n][0], s[mt][n][1]);
            f2_split(f2_mul(f2_make(p2, p3), f2_make(vb, vb)), s[mt][n][2], s[mt][n][3]);
            top[n][0] = fmax3(top[n][0], s[mt][n][0], s[mt][n][2]);
            top[n][1] = fmax3(top[n][1], s[mt][n][1], s[mt][n][3]);
        }
    }
    uint32_t pb[MTS][NT][2];
    uint64_t back[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        // the exponents alone, two columns in a word (both are positive)
        uint32_t t = __byte_perm(__float_as_uint(top[n][0]), __float_as_uint(top[n][1]), 0x7632);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
            t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
        const uint32_t e0 = max(t >> 7 & 0xffu, 15u), e1 = max(t >> 23, 15u);  // 2^(e - 127), or 2^-112
        const uint64_t f = f2_make(__uint_as_float((268 - e0) << 23), __uint_as_float((268 - e1) << 23));
        back[n] = f2_make(__uint_as_float((e0 - 14) << 23), __uint_as_float((e1 - 14) << 23));
#pragma unroll
        for (int mt = 0; mt < MTS; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // keys 0-7 of the 16, keys 8-15
                float x0, x1;
                f2_split(f2_mul(f2_make(s[mt][n][2 * e], s[mt][n][2 * e + 1]), f), x0, x1);
                pb[mt][n][e] = movmatrix_trans(pack_f16(x0, x1));
            }
    }
#pragma unroll
    for (int dt = 0; dt < kD / 16; ++dt) {
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        const int da = dt * 16 + g, db = da + 8;
#pragma unroll
        for (int mt = 0; mt < MTS; ++mt) {
            uint32_t wa = *reinterpret_cast<const uint32_t *>(sV + da * 64 + ((mt ^ ((da >> 1) & 3)) << 4) + 4 * tq);
            uint32_t wb = *reinterpret_cast<const uint32_t *>(sV + db * 64 + ((mt ^ ((db >> 1) & 3)) << 4) + 4 * tq);
            if (PART) {
                // a thread's word holds the codes of keys 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9 of the 16
                const int k0 = mt * 16 + 2 * tq;
                const uint32_t mask = (k0 < valid ? 0xffu : 0u) | (k0 + 1 < valid ? 0xff00u : 0u) |
                                      (k0 + 8 < valid ? 0xff0000u : 0u) | (k0 + 9 < valid ? 0xff000000u : 0u);
                wa &= mask;
                wb &= mask;
            }
            const uint32_t a[4] = {fp8x2_lo<E5M2>(wa), fp8x2_lo<E5M2>(wb), fp8x2_hi<E5M2>(wa),
                                   fp8x2_hi<E5M2>(wb)};
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma_f16_16816(acc[n], a, pb[mt][n][0], pb[mt][n][1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; e += 2)  // rows 2 tq, 2 tq + 1 of dimension da, then of db
                f2_split(f2_fma(f2_make(acc[n][e], acc[n][e + 1]), back[n], f2_make(st.o[dt][n][e], st.o[dt][n][e + 1])),
                         st.o[dt][n][e], st.o[dt][n][e + 1]);
    }
}

// Q as the B operand: column g of n-tile n is row col0 + 8 n + g (zero past G T).  F16: for an FP8
// page, whose codes are exact in fp16 (so is q between 2^-14 and 65504).
template <int NT, bool F16>
__device__ __forceinline__ void load_q(const WeighParams &p, int b, int h, int col0, int lane,
                                       uint32_t (&qb)[NT][kD / 16][2])
{
    const int g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = col0 + n * 8 + g;
        const bool ok = row < p.G * p.T;
        const int t = ok ? row / p.G : 0, hh = ok ? row % p.G : 0;
        const __nv_bfloat16 *q = p.q + (((int64_t)b * p.T + t) * (p.G * p.Hkv) + h * p.G + hh) * kD + 2 * tq;
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w = ok ? __ldg(reinterpret_cast<const uint32_t *>(q + ks * 16 + 8 * e)) : 0u;
                qb[n][ks][e] = F16 ? bf16x2_to_f16x2(w) : w;
            }
    }
}

template <int FP8, int NT, int RH>
__global__ void __launch_bounds__(Shape<FP8, NT, RH>::kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const WeighParams p)
{
    using S = Shape<FP8, NT, RH>;
    constexpr int kThr = S::kThreads, NS = S::kStages, GW = S::kGroups, CW = S::kWarps;
    constexpr int RP = 8 * NT * RH;
    extern __shared__ uint8_t smem_raw[];
    AttendSmem<FP8, NT, RH> &sh = *reinterpret_cast<AttendSmem<FP8, NT, RH> *>(align_smem_1024(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], RH);
        }
        fence_barrier_init();
    }
    if (warp == CW && lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- this CTA's contiguous range of pages ---------------------------------------------
    const int per = (p.B + kThr - 1) / kThr;
    const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
    int local = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int c = seq_len(p, b);
        if (b < kLens)
            sh.len[b] = c;
        if (c < 0 && blockIdx.x == 0)
            set_err(p.dev_err, HSA_DEVERR_BAD_LEN);
        local += pages_of(c);
    }
    const int64_t N = (int64_t)block_scan<kThr>(sh.scan, &sh.total, local, tid) * p.Hkv;
    const int64_t C = N < (int64_t)gridDim.x ? N : (int64_t)gridDim.x;
    if ((int64_t)blockIdx.x >= C)
        return;
    const int64_t i0 = (int64_t)blockIdx.x * N / C, i1 = ((int64_t)blockIdx.x + 1) * N / C;
    auto length = [&](int b) { return b < kLens ? sh.len[b] : seq_len(p, b); };
    {
        int before = sh.scan[tid];
        for (int b = b_lo; b < b_hi; ++b) {
            const int n = pages_of(length(b));
            if ((int64_t)(before + n) * p.Hkv > i0 && (int64_t)before * p.Hkv <= i0) {
                sh.first_b = b;
                sh.before = before;
            }
            before += n;
        }
    }
    __syncthreads();
    UnitWalk w0;
    w0.b = sh.first_b;
    w0.c = length(w0.b);
    w0.n = pages_of(w0.c);
    {
        const int64_t off = i0 - (int64_t)sh.before * p.Hkv;
        w0.h = (int)(off / w0.n);
        w0.j = (int)(off % w0.n);
    }
    auto next = [&](UnitWalk &w) {
        if (++w.j < w.n)
            return;
        w.j = 0;
        if (++w.h < p.Hkv)
            return;
        w.h = 0;
        do {  // past sequences that are left out
            if (++w.b >= p.B)
                return;
            w.c = length(w.b);
            w.n = pages_of(w.c);
        } while (w.n == 0);
    };

    if (warp == CW) {
        // ------------------------------------------------------------------------ producer
        // lane l finds the pool row of page start + l, 32 pages at a time and a batch ahead; the
        // whole warp waits for the stages and one elected lane issues them
        if (kWithholdLoads)
            return;
        const uint64_t pol = policy_evict_first();
        const int64_t cb = fp8_codes_bytes(p.num_blocks, p.Hkv);
        auto pool_row = [&](const UnitWalk &w) -> int64_t {
            if (w.c == 0)
                return -1;
            if (w.j >= p.max_blocks) {
                set_err(p.dev_err, HSA_DEVERR_BAD_PAGE);
                return -1;
            }
            const int blk = __ldg(p.block_tables + (int64_t)w.b * p.max_blocks + w.j);
            if (blk < 0 || blk >= p.num_blocks) {
                set_err(p.dev_err, HSA_DEVERR_BAD_BLOCK);
                return -1;
            }
            return ((int64_t)blk * p.Hkv + w.h) * kTileKeys;
        };
        UnitWalk wl = w0;
        int64_t row = -1;
        if (i0 + lane < i1) {
            for (int e = 0; e < lane; ++e)
                next(wl);
            row = pool_row(wl);
        }
        int64_t k = 0;
        bool stop = false;
        for (int64_t ib = i0; ib < i1 && !stop; ib += 32) {
            int64_t nrow = -1;
            if (ib + 32 + lane < i1) {
                for (int e = 0; e < 32; ++e)
                    next(wl);
                nrow = pool_row(wl);
            }
            const int cnt = (int)(i1 - ib < 32 ? i1 - ib : 32);
            for (int e = 0; e < cnt; ++e, ++k) {
                const int64_t r = __shfl_sync(0xffffffffu, row, e);
                const int st = (int)(k % NS);
                if (!__all_sync(0xffffffffu, mbar_wait(&sh.empty[st], (uint32_t)((k / NS) & 1) ^ 1))) {
                    if (lane == 0)
                        set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
                    stop = true;
                    break;
                }
                uint8_t *const dst = sh.stage + st * S::kStageStride;
                if (elect_one()) {
                    sh.tile_ok[st] = r >= 0;
                    if (r < 0) {
                        mbar_arrive(&sh.full[st]);
                    } else if (FP8) {
                        mbar_arrive_expect_tx(&sh.full[st], 2 * kFp8TileBytes + 2 * 256);
                        tma_load_2d(dst, &tmK, &sh.full[st], 0, (int32_t)r, pol);
                        tma_load_2d(dst + kFp8TileBytes, &tmV, &sh.full[st], 0, (int32_t)(2 * r), pol);
                        bulk_load(dst + 2 * kFp8TileBytes, reinterpret_cast<const uint8_t *>(p.k_pool) + cb + r * 4, 256,
                                  &sh.full[st], pol);
                        bulk_load(dst + 2 * kFp8TileBytes + 256, reinterpret_cast<const uint8_t *>(p.v_pool) + cb + r * 4,
                                  256, &sh.full[st], pol);
                    } else {
                        mbar_arrive_expect_tx(&sh.full[st], 2 * kTileBytes);
                        tma_load_2d(dst, &tmK, &sh.full[st], 0, (int32_t)r, pol);
                        tma_load_2d(dst + kTileBytes / 2, &tmK, &sh.full[st], 64, (int32_t)r, pol);
                        tma_load_2d(dst + kTileBytes, &tmV, &sh.full[st], 0, (int32_t)r, pol);
                        tma_load_2d(dst + kTileBytes + kTileBytes / 2, &tmV, &sh.full[st], 64, (int32_t)r, pol);
                    }
                }
                __syncwarp();
            }
            row = nrow;
        }
        if (lane == 0) {
            // no copy may still be in flight when the CTA exits
            for (int64_t s = 0; s < NS && s < k; ++s) {
                const int64_t last = s + ((k - 1 - s) / NS) * NS;
                mbar_wait(&sh.full[s], (uint32_t)((last / NS) & 1));
            }
        }
        return;
    }

    // ---------------------------------------------------------------------------- consumers
    const int group = warp / RH, rh = warp % RH, col0 = rh * 8 * NT;
    const int g = lane >> 2, tq = lane & 3;
    State<NT> st;
    uint32_t qb[NT][kD / 16][2];
    UnitWalk w = w0;
    bool fresh = true, used = false, timed_out = false;
    for (int64_t i = i0, k = 0; i < i1; ++i, ++k) {
        const int64_t unit = (int64_t)w.b * p.Hkv + w.h;
        float *const score = p.score + unit * p.w_stride * p.srow;
        if (fresh) {
            fresh = used = false;
            clear(st);
            load_q<NT, FP8 != 0>(p, w.b, w.h, col0, lane, qb);
        }
        if ((int)(k % GW) == group) {
            const int stg = (int)(k % NS);
            if (!timed_out && !mbar_wait(&sh.full[stg], (uint32_t)((k / NS) & 1))) {
                set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
                timed_out = true;
            }
            const int valid = min(kTileKeys, w.c - w.j * kTileKeys);  // cached keys of the page
            float *const to = score + (int64_t)w.j * kTileKeys * p.srow;
            if (!timed_out && valid > 0 && sh.tile_ok[stg] != 0) {
                used = true;
                uint8_t *const base = sh.stage + stg * S::kStageStride;
                if constexpr (FP8 != 0) {
                    const float *ks = reinterpret_cast<const float *>(base + 2 * kFp8TileBytes);
                    if (valid == kTileKeys)
                        tile_fp8<NT, FP8 == 2, false>(st, qb, base, base + kFp8TileBytes, ks, ks + 64, valid, col0,
                                                      p.scale_log2, to, p.srow, lane);
                    else
                        tile_fp8<NT, FP8 == 2, true>(st, qb, base, base + kFp8TileBytes, ks, ks + 64, valid, col0,
                                                     p.scale_log2, to, p.srow, lane);
                } else {
                    if (valid < kTileKeys) {
                        // rows of V past the last token meet zero weights: whatever the page
                        // holds there must not
                        for (int e = valid * 16 + lane; e < kTileKeys * 16; e += 32)
                            *reinterpret_cast<uint4 *>(base + kTileBytes + swz128_offset(e >> 4, (e & 15) * 8, kTileKeys)) =
                                make_uint4(0, 0, 0, 0);
                        __syncwarp();
                    }
                    tile_bf16<NT, kTileKeys / 16>(st, qb, smem_u32(base), smem_u32(base) + kTileBytes, kTileKeys, valid,
                                                  false, p.G, col0, p.scale_log2, to, p.srow, lane);
                    if (valid < kTileKeys)
                        fence_proxy_async_smem();  // the zeros, before the stage's next copy
                }
            } else if (valid > 0 && rh == 0) {  // absent keys
                for (int e = lane; e < valid * p.srow; e += 32)
                    to[e] = -INFINITY;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.empty[stg]);
        }
        const bool last_page = w.j == w.n - 1;
        if (!last_page && i != i1 - 1) {
            next(w);
            continue;
        }
        // ---- the end of the unit, or of this CTA's part of it ------------------------------
        if constexpr (FP8 != 0) {  // fp16 roundings (tile_fp8): 2^-11 of a weight, the sum does without
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    st.lr[n][e] = st.l[n][e];
        }
        if (last_page && group == 0) {
            // the new tokens: rows >= T of the tile are zero
            used = true;
            if constexpr (FP8 != 0)
                load_q<NT, false>(p, w.b, w.h, col0, lane, qb);
            for (int e = lane; e < kNewKeys * 16; e += 32) {
                const int t = e >> 4, ch = e & 15;
                uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
                if (t < p.T) {
                    const int64_t at = (((int64_t)w.b * p.T + t) * p.Hkv + w.h) * 16 + ch;
                    kv = __ldg(reinterpret_cast<const uint4 *>(p.k_new) + at);
                    vv = __ldg(reinterpret_cast<const uint4 *>(p.v_new) + at);
                }
                *reinterpret_cast<uint4 *>(sh.new_k[rh] + swz128_offset(t, ch * 8, kNewKeys)) = kv;
                *reinterpret_cast<uint4 *>(sh.new_v[rh] + swz128_offset(t, ch * 8, kNewKeys)) = vv;
            }
            __syncwarp();
            tile_bf16<NT, 1>(st, qb, smem_u32(sh.new_k[rh]), smem_u32(sh.new_v[rh]), kNewKeys, p.T, true, p.G, col0,
                             p.scale_log2, score + (int64_t)w.c * p.srow, p.srow, lane);
            __syncwarp();
        }
        float *const part = p.part + ((unit + blockIdx.x) * GW + group) * slot_floats(RP);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = st.l[n][e], lr = st.lr[n][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    l += __shfl_xor_sync(0xffffffffu, l, o);
                    lr += __shfl_xor_sync(0xffffffffu, lr, o);
                }
                const int row = col0 + n * 8 + 2 * tq + e;
                if (g == 0) {
                    part[row] = st.m[n][e];
                    part[RP + row] = l;
                    part[2 * RP + row] = used ? lr : kUnused;
                }
            }
        if (used) {
            float *const po = part + 3 * RP;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float *const to = po + (col0 + n * 8 + 2 * tq) * kD + g;
#pragma unroll
                for (int dt = 0; dt < kD / 16; ++dt) {
                    to[dt * 16] = st.o[dt][n][0];
                    to[kD + dt * 16] = st.o[dt][n][1];
                    to[dt * 16 + 8] = st.o[dt][n][2];
                    to[kD + dt * 16 + 8] = st.o[dt][n][3];
                }
            }
        }
        fresh = true;
        next(w);
    }
}

// The T new rows of unit (b, h) into the layer.
__device__ __forceinline__ void append_rows(const WeighParams &p, int b, int h, int c, int tid)
{
    const int lane = tid & 31;
    auto page_row = [&](int t, int *blk_out) -> int64_t {
        const int64_t pos = (int64_t)c + t;
        if (pos / kTileKeys >= p.max_blocks) {
            set_err(p.dev_err, HSA_DEVERR_BAD_PAGE);
            return -1;
        }
        const int blk = __ldg(p.block_tables + (int64_t)b * p.max_blocks + pos / kTileKeys);
        if (blk < 0 || blk >= p.num_blocks) {
            set_err(p.dev_err, HSA_DEVERR_BAD_BLOCK);
            return -1;
        }
        *blk_out = blk;
        return ((int64_t)blk * p.Hkv + h) * kTileKeys + pos % kTileKeys;
    };
    if (p.fp8) {
        for (int e = tid >> 5; e < 2 * p.T; e += kJoinThreads / 32) {
            const int kv = e & 1, t = e >> 1;
            int blk = 0;
            if (page_row(t, &blk) < 0)
                continue;
            uint8_t *codes = reinterpret_cast<uint8_t *>(kv ? p.v_pool : p.k_pool);
            fp8_store_row((kv ? p.v_new : p.k_new) + (((int64_t)b * p.T + t) * p.Hkv + h) * kD, codes,
                          reinterpret_cast<float *>(codes + fp8_codes_bytes(p.num_blocks, p.Hkv)), blk, h, p.Hkv,
                          (int)(((int64_t)c + t) % kTileKeys), kv, lane, p.fp8 == 2);
        }
        return;
    }
    for (int e = tid; e < 32 * p.T; e += kJoinThreads) {
        const int t = e >> 5, kv = (e >> 4) & 1, ch = e & 15;
        int blk = 0;
        const int64_t row = page_row(t, &blk);
        if (row >= 0)
            (kv ? p.v_pool : p.k_pool)[row * 16 + ch] =
                __ldg(reinterpret_cast<const uint4 *>(kv ? p.v_new : p.k_new) +
                      (((int64_t)b * p.T + t) * p.Hkv + h) * 16 + ch);
    }
}

constexpr int kMaxParts = 2048;                  // groups of all CTAs (152 x 8; launch_attend)

struct JoinSmem {
    int32_t len[kLens];
    int32_t scan[kJoinThreads];
    float m[kMaxRows], lse[kMaxRows], norm[kMaxRows];
    int32_t list[kMaxParts];  // the unit's states that hold keys
    int32_t listed[kJoinThreads / 32];
    int32_t first_b, before, total;
    int32_t pages_total, pages_before;
};

// VEC scores a load, LK lanes a key: srow = VEC LK.  GW: groups of the attend kernel, RP its padded
// rows, ctas its grid.
template <int VEC, int LK>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtas)
    join_kernel(const WeighParams p, int GW, int RP, int ctas)
{
    constexpr int kStep = kJoinThreads / LK, kChunk = kBatch * kStep;  // positions an item
    __shared__ JoinSmem sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // (the lengths are no work of the attend kernel's, which itself waited for what was queued before
    // it: this CTA's range is found meanwhile.  few 20.4 -> 18.4 us, verify 120 -> 118)
    const int rows = p.G * p.T, out_items = (rows + 7) / 8;
    auto items_of = [&](int c) { return c < 0 ? 0 : out_items + (c + p.T + kChunk - 1) / kChunk; };
    const int per = (p.B + kJoinThreads - 1) / kJoinThreads;
    const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
    auto length = [&](int b) { return b < kLens ? sh.len[b] : seq_len(p, b); };
    int local = 0, pages = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int c = seq_len(p, b);
        if (b < kLens)
            sh.len[b] = c;
        local += items_of(c);
        pages += pages_of(c);
    }
    const int64_t PN = (int64_t)block_scan<kJoinThreads>(sh.scan, &sh.pages_total, pages, tid) * p.Hkv;
    const int pages_before = sh.scan[tid];
    __syncthreads();
    const int64_t N = (int64_t)block_scan<kJoinThreads>(sh.scan, &sh.total, local, tid) * p.Hkv;
    const int64_t C = N < (int64_t)gridDim.x ? N : (int64_t)gridDim.x;
    if ((int64_t)blockIdx.x >= C) {
        grid_dependency_wait();  // no end of this grid before the attend kernel's
        return;
    }
    const int64_t i0 = (int64_t)blockIdx.x * N / C, i1 = ((int64_t)blockIdx.x + 1) * N / C;
    {
        int before = sh.scan[tid], pb = pages_before;
        for (int b = b_lo; b < b_hi; ++b) {
            const int n = items_of(length(b));
            if ((int64_t)(before + n) * p.Hkv > i0 && (int64_t)before * p.Hkv <= i0) {
                sh.first_b = b;
                sh.before = before;
                sh.pages_before = pb;
            }
            before += n;
            pb += pages_of(length(b));
        }
    }
    __syncthreads();
    grid_dependency_wait();
    int b = sh.first_b, c = length(b), n = items_of(c);
    int64_t pb = sh.pages_before;
    const int64_t off = i0 - (int64_t)sh.before * p.Hkv;
    int h = (int)(off / n), j = (int)(off % n);
    const int64_t PC = PN < (int64_t)ctas ? PN : (int64_t)ctas;
    bool fresh = true;
    const float *part = nullptr;
    int parts = 0;
    float lse[VEC];
    const int sub = tid % LK;
    for (int64_t i = i0; i < i1; ++i) {
        const int64_t unit = (int64_t)b * p.Hkv + h;
        if (fresh) {
            fresh = false;
            // the unit's states: those of every CTA whose range met its pages, side by side
            const int np = pages_of(c);
            const int64_t u0 = pb * p.Hkv + (int64_t)h * np, u1 = u0 + np;
            const int64_t c_lo = ((u0 + 1) * PC - 1) / PN, c_hi = (u1 * PC - 1) / PN;
            part = p.part + (unit + c_lo) * GW * slot_floats(RP);
            parts = (int)(c_hi - c_lo + 1) * GW;
            __syncthreads();  // the last unit's readers are done
            // of a few pages a CTA, most groups have none: their states are left out
            int held = 0;
            for (int e0 = 0; e0 < parts; e0 += kJoinThreads) {
                const int e = e0 + tid;
                const bool on = e < parts && __ldcg(part + (int64_t)e * slot_floats(RP) + 2 * RP) != kUnused;
                const uint32_t bits = __ballot_sync(0xffffffffu, on);
                if (lane == 0)
                    sh.listed[warp] = __popc(bits);
                __syncthreads();
                int at = held + __popc(bits & ((1u << lane) - 1));
                for (int w = 0; w < kJoinThreads / 32; ++w) {
                    at += w < warp ? sh.listed[w] : 0;
                    held += sh.listed[w];
                }
                if (on)
                    sh.list[at] = e;
                __syncthreads();
            }
            parts = held;
            const int row = tid >> 3, s8 = tid & 7;  // eight threads a row
            float M = -INFINITY, L = 0.f, R = 0.f;
            constexpr int kAhead = 4;
            for (int e0 = s8; row < rows && e0 < parts; e0 += 8 * kAhead) {
                float m[kAhead], l[kAhead], r[kAhead], top = M;
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    const bool on = e0 + 8 * e < parts;
                    const float *q = part + (int64_t)sh.list[on ? e0 + 8 * e : 0] * slot_floats(RP) + row;
                    m[e] = on ? __ldcg(q) : -INFINITY;
                    l[e] = on ? __ldcg(q + RP) : 0.f;
                    r[e] = on ? __ldcg(q + 2 * RP) : 0.f;
                }
#pragma unroll
                for (int e = 0; e < kAhead; ++e)
                    top = fmaxf(top, m[e]);
                const float base = top == -INFINITY ? 0.f : top, f = fast_exp2(M - base);
                L *= f;
                R *= f;
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    const float a = fast_exp2(m[e] - base);
                    L += l[e] * a;
                    R += r[e] * a;
                }
                M = top;
            }
            float top = M;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float base = top == -INFINITY ? 0.f : top, f = fast_exp2(M - base);
            L *= f;
            R *= f;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                L += __shfl_xor_sync(0xffffffffu, L, o);
                R += __shfl_xor_sync(0xffffffffu, R, o);
            }
            if (s8 == 0) {
                sh.m[row] = base;
                sh.lse[row] = row < rows && L != 0.f ? base + log2f(L) : INFINITY;  // (NaN passes)
                sh.norm[row] = R > 0.f ? 1.f / R : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                lse[e] = sh.lse[sub * VEC + e];
        }
        if (j < out_items) {
            // ---- eight rows of output, a warp each, four dimensions a lane ------------------
            const int row = j * 8 + warp;
            if (row < rows) {
                const float base = sh.m[row];
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                constexpr int kAhead = 8;
                for (int e0 = 0; e0 < parts; e0 += kAhead) {
                    float m[kAhead];
                    float4 x[kAhead];
#pragma unroll
                    for (int e = 0; e < kAhead; ++e) {
                        const bool on = e0 + e < parts;
                        const float *q = part + (int64_t)sh.list[on ? e0 + e : 0] * slot_floats(RP);
                        m[e] = on ? __ldcg(q + row) : -INFINITY;
                        x[e] = on ? __ldcg(reinterpret_cast<const float4 *>(q + 3 * RP + row * kD) + lane)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int e = 0; e < kAhead; ++e) {
                        const float a = fast_exp2(m[e] - base);
                        acc.x += x[e].x * a;
                        acc.y += x[e].y * a;
                        acc.z += x[e].z * a;
                        acc.w += x[e].w * a;
                    }
                }
                const float f = sh.norm[row];
                const int t = row / p.G, hh = row % p.G;
                *reinterpret_cast<uint2 *>(
                    p.out + (((int64_t)b * p.T + t) * (p.G * p.Hkv) + h * p.G + hh) * kD + 4 * lane) =
                    make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
            }
            if (j == 0 && p.append)
                append_rows(p, b, h, c, tid);
        } else {
            // ---- the weights of the unit's positions in this CTA's range ----------------------
            // kBatch positions a thread are on the way all the time: the next ones' loads go out as
            // each is used, ahead of its store (which might be to the same weights)
            const int items = (int)min((int64_t)(n - j), i1 - i);
            const int first = (j - out_items) * kChunk, end = min(c + p.T, first + items * kChunk);
            const float *const score = p.score + unit * p.w_stride * p.srow;
            const int64_t at = unit * p.w_stride;
            float4 x[kBatch];
            float old[kBatch];
            auto fetch = [&](int k, int pos) {
                x[k] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                old[k] = 0.f;
                if (pos < end) {
                    const float *s = score + (int64_t)pos * p.srow + sub * VEC;
                    if constexpr (VEC == 4) {
                        x[k] = __ldcg(reinterpret_cast<const float4 *>(s));
                    } else {
                        const float2 y = __ldcg(reinterpret_cast<const float2 *>(s));
                        x[k].x = y.x;
                        x[k].y = y.y;
                    }
                    if (sub == 0 && p.w_prev && pos < c)
                        old[k] = p.w_prev[at + pos];
                }
            };
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                fetch(k, first + tid / LK + k * kStep);
            for (int p0 = first; p0 < end; p0 += kChunk) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int pos = p0 + tid / LK + k * kStep;
                    const float4 y = x[k];
                    const float before = old[k];
                    fetch(k, pos + kChunk);
                    float sum = fast_exp2(y.x - lse[0]) + fast_exp2(y.y - lse[1]);
                    if constexpr (VEC == 4)
                        sum += fast_exp2(y.z - lse[2]) + fast_exp2(y.w - lse[3]);
#pragma unroll
                    for (int o = 1; o < LK; o <<= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (pos < end && sub == 0)
                        p.w[at + pos] = p.w_prev && pos < c ? fmaf(p.decay, before, sum) : sum;
                }
            }
            i += items - 1;
            j += items - 1;
        }
        if (++j < n)
            continue;
        j = 0;
        fresh = true;
        if (++h < p.Hkv)
            continue;
        h = 0;
        do {
            pb += pages_of(c);
            if (++b >= p.B)
                break;
            c = length(b);
            n = items_of(c);
        } while (n == 0);
    }
}

int score_rows(int rows)
{
    int s = 2;
    while (s < rows)
        s *= 2;
    return s;
}

template <int FP8, int NT, int RH>
cudaError_t launch_attend(const CUtensorMap &tmK, const CUtensorMap &tmV, const WeighParams &p, int ctas,
                          int join_ctas, cudaStream_t stream)
{
    using S = Shape<FP8, NT, RH>;
    const size_t smem = sizeof(AttendSmem<FP8, NT, RH>) + 1024;
    ctas = ctas < kMaxParts / S::kGroups ? ctas : kMaxParts / S::kGroups;
    static SmemOptIn opt;
    cudaError_t e = opt.set(attend_kernel<FP8, NT, RH>, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend_kernel<FP8, NT, RH>, tmK, tmV, p);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3((unsigned)join_ctas);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    void (*join)(WeighParams, int, int, int) = p.srow == 2   ? join_kernel<2, 1>
                                               : p.srow == 4  ? join_kernel<4, 1>
                                               : p.srow == 8  ? join_kernel<4, 2>
                                               : p.srow == 16 ? join_kernel<4, 4>
                                                              : join_kernel<4, 8>;
    return cudaLaunchKernelEx(&cfg, join, p, S::kGroups, 8 * NT * RH, ctas);
}

template <int FP8>
cudaError_t launch_rows(const CUtensorMap &tmK, const CUtensorMap &tmV, const WeighParams &p, int ctas,
                        int join_ctas, cudaStream_t stream)
{
    const int rows = p.G * p.T;
    return rows <= 8    ? launch_attend<FP8, 1, 1>(tmK, tmV, p, ctas, join_ctas, stream)
           : rows <= 16 ? launch_attend<FP8, 2, 1>(tmK, tmV, p, ctas, join_ctas, stream)
                        : launch_attend<FP8, 2, 2>(tmK, tmV, p, ctas, join_ctas, stream);
}

}  // namespace

WeighLayout weigh_layout(int ctas, int B, int T, int G, int Hkv, int w_stride)
{
    const int rows = G * T, padded = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
    const size_t slots = ((size_t)B * Hkv + ctas) * 8;  // at most eight groups a CTA
    WeighLayout lay;
    lay.part = 0;
    lay.score = (slots * slot_floats(padded) * sizeof(float) + 255) & ~size_t(255);
    lay.total = lay.score + (size_t)B * Hkv * w_stride * score_rows(rows) * sizeof(float);
    return lay;
}

cudaError_t launch_weigh(const CUtensorMap &tmK, const CUtensorMap &tmV, const WeighParams &params, int sms,
                         int max_ctas, cudaStream_t stream)
{
    const int most = max_ctas > 0 ? max_ctas : INT32_MAX;  // of each launch
    const int ctas = sms < most ? sms : most, join_ctas = kJoinCtas * sms < most ? kJoinCtas * sms : most;
    WeighParams p = params;
    p.srow = score_rows(p.G * p.T);
    return p.fp8 == 2   ? launch_rows<2>(tmK, tmV, p, ctas, join_ctas, stream)
           : p.fp8 == 1 ? launch_rows<1>(tmK, tmV, p, ctas, join_ctas, stream)
                        : launch_rows<0>(tmK, tmV, p, ctas, join_ctas, stream);
}

}  // namespace hsa

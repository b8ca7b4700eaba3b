// rope.cu -- rotary positions on several axes, alone and on the way into the dual KV
// pool (sm_103a).
//
// What it computes: for token n, a query or key head x[0 .. d-1] and pair i of its first
// rot_dim values, (a, b) = (i, i + rot_dim / 2) or (2 i, 2 i + 1),
//   y_a = s (x_a cos t - x_b sin t),  y_b = s (x_b cos t + x_a sin t),
//   t = pos[axis(i)][n] * inv_freq[i],
// values past rot_dim unchanged.  Several axes (time, height, width) give an image's or
// a video's tokens a position on each [youleyou.com "小米MiMo首次公开模型推理系统全链路优化
// 降价99%", s2 "Decode加速与多模态优化": the stack serves images and video].  The append
// form also writes the turned keys and the values where hsa_kv_append would: a page row of
// a full layer (bf16, or FP8 codes and a scale), or a ring slot.
//
// The angle: an fp32 product pos * inv_freq is off by 2^-24 of itself, 0.06 rad at a
// million tokens.  Only its fraction of a turn matters, so the host gives inv_freq / 2 pi
// as a 64-bit binary fraction F of a turn and the kernel takes the low 64 bits of
// pos * F: the whole turns fall off the top, exactly, and the top 32 bits are the angle
// to 2^-31 of a turn for every 32-bit position, negative ones too.  One integer
// multiply; cos and sin then see an fp32 argument in [-1, 1] half turns, whose rounding is
// 2^-26 of a turn at most.
//
// Layout: eight lanes take a head, lane c its 16-byte chunks c and c + rot_dim / 16, which
// hold both sides of each of its eight pairs (or, interleaved, eight whole pairs), so a
// pair never crosses lanes; chunks past rot_dim go to the remaining lanes.  A warp takes
// four heads at a time and reads 128 contiguous bytes of each.  Each lane computes two of
// a token's 64 angles and the warp exchanges them by shuffles, once for all heads.
//
// What bounds it: the reads and writes, each head once (measured copy 6.8 TB/s): 20011 tokens
// of 32 / 4 heads in 60 us, 6.2 TB/s; with the pool 34985 tokens in 121 us, 6.2 TB/s; a ring,
// whose 128 rows a request are few of the 7897, 29 us, 5.2 TB/s.  Five head quads in flight
// a warp and two blocks an SM: ten quads or three blocks were no faster.  An FP8 layer is bound
// by latency: 7447 tokens take 43 us, 3.5 TB/s, with 28% of the DRAM's cycles in use and
// instructions (divisions, codes, the transposed V; 20 million) issued in 48%, as 16 warps an SM
// wait for their loads and for each other's results, and as the last of a warp's four items
// leaves others idle.  32 tokens take 2.4 us alone and 3.5 with the pool, less than the host's
// call.
#include "fp8_kv.cuh"
#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 5;  // head quads whose loads are in flight together
constexpr int kBlocks = 2; // blocks an SM

enum Kind { kRope = 0, kAppend = 1, kAppendFp8 = 2 };

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8])
{
    x[0] = bf16_lo(w.x);
    x[1] = bf16_hi(w.x);
    x[2] = bf16_lo(w.y);
    x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z);
    x[5] = bf16_hi(w.z);
    x[6] = bf16_lo(w.w);
    x[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

// The eight pairs of a lane's two chunks turned by (cs, sn) j = 0 .. 7.
template <bool INTER>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&cs)[8],
                                     const float (&sn)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float &x = INTER ? (j < 4 ? a[2 * j] : b[2 * (j - 4)]) : a[j];
        float &y = INTER ? (j < 4 ? a[2 * j + 1] : b[2 * (j - 4) + 1]) : b[j];
        const float x0 = x, y0 = y;
        x = x0 * cs[j] - y0 * sn[j];
        y = y0 * cs[j] + x0 * sn[j];
    }
}

// Request that owns token tok: the r with cu[r] <= tok < cu[r + 1], by a 32-way search (one
// coalesced read a level, not log2 R dependent ones).  Called by a whole warp.
__device__ __forceinline__ int find_request(const int32_t *cu, int R, int tok, int lane)
{
    int lo = 0, hi = R;  // cu[lo] <= tok (or lo = 0), tok < cu[hi] (or hi = R)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int at = lo + (lane + 1) * step;  // candidates lo + step, lo + 2 step, ...
        const bool le = at < hi && __ldg(cu + at) <= tok;
        const int k = __popc(__ballot_sync(0xffffffffu, le));
        const int nlo = lo + k * step;
        hi = min(hi, nlo + step);
        lo = nlo;
    }
    return lo;
}

// Destination row of cache position pos of sequence seq (units of one head's rows), or
// -1 with *err set.  (A start and an offset of 31 bits each: the sum has 32.)
__device__ __forceinline__ int64_t pool_row(const RopeParams &p, int seq, uint32_t pos, int *err)
{
    if (seq < 0 || seq >= p.batch) {
        *err = HSA_DEVERR_BAD_SEQ;
        return -1;
    }
    if (p.ring_mode) {
        const int rr = __ldg(p.ring_row + seq);
        if (rr < 0 || rr >= p.n_ring_rows) {
            *err = HSA_DEVERR_BAD_RING;
            return -1;
        }
        return (int64_t)rr * p.Hkv * p.W + pos % (uint32_t)p.W;
    }
    const uint32_t page = pos / 64;
    if (page >= (uint32_t)p.max_blocks) {
        *err = HSA_DEVERR_BAD_PAGE;
        return -1;
    }
    const int blk = __ldg(p.block_tables + (int64_t)seq * p.max_blocks + page);
    if (blk < 0 || blk >= p.num_blocks) {
        *err = HSA_DEVERR_BAD_BLOCK;
        return -1;
    }
    return (int64_t)blk * p.Hkv * 64 + pos % 64;
}

// One FP8 row a lane octet: a, b the lane's chunks ca, cb of the head in fp32 (quantised
// straight from them: one rounding).  K rows go through `stage` (128 bytes of shared memory
// an octet) into 16-byte stores; V rows are stored transposed, a byte a dimension.
__device__ __forceinline__ void store_fp8(const float (&a)[8], const float (&b)[8], int ca, int cb,
                                          bool on, bool is_v, int64_t row, int h,
                                          const RopeParams &p, uint8_t *stage, int c)
{
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        amax = fmaxf(amax, fmaxf(fabsf(a[j]), fabsf(b[j])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const bool e5 = p.fp8 == 2;
    const float scale = __fdiv_rn(amax, e5 ? 57344.0f : 448.0f);
    uint32_t code[8];  // two codes each: a's four pairs of neighbours, then b's
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = j < 4 ? a[2 * j] : b[2 * j - 8], y = j < 4 ? a[2 * j + 1] : b[2 * j - 7];
        code[j] = 0;
        if (amax > 0.f) {
            const float u = __fdiv_rn(x, scale), w = __fdiv_rn(y, scale);
            code[j] = e5 ? f32x2_to_e5m2x2(u, w) : f32x2_to_e4m3x2(u, w);
        }
    }
    // row = blk * Hkv * 64 + off: head h's page is blk * Hkv + h
    const int off = (int)(row & 63);
    const int64_t page = (row >> 6) + h;
    uint8_t *const base = reinterpret_cast<uint8_t *>(is_v ? p.v_dst : p.k_dst);
    float *const scales = reinterpret_cast<float *>(base + fp8_codes_bytes(p.num_blocks, p.Hkv));
    if (on && c == 0)
        scales[page * 64 + off] = amax > 0.f ? scale : 0.f;
    if (!is_v) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int ch = j < 4 ? ca : cb;  // dims 8 ch + 2 (j % 4), +1
            *reinterpret_cast<uint16_t *>(stage + 16 * (ch >> 1) + 2 * (ch & 1) + 4 * (j & 3)) =
                (uint16_t)code[j];
        }
        __syncwarp();
        if (on)
            *reinterpret_cast<uint4 *>(base + (page * 64 + off) * 128 + 16 * c) =
                *reinterpret_cast<const uint4 *>(stage + 16 * c);
    } else if (on) {
        const int kb = 16 * (off >> 4) + perm16(off & 15);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int dim = 8 * (j < 4 ? ca : cb) + 2 * (j & 3);
            base[(page * 128 + dim) * 64 + kb] = (uint8_t)code[j];
            base[(page * 128 + dim + 1) * 64 + kb] = (uint8_t)(code[j] >> 8);
        }
    }
}

// Values of an FP8 layer, 16 keys of one KV head at a time.  V pages are stored transposed (64
// bytes of keys a dimension), so a token on its own is 128 single-byte stores, each a 32-byte
// sector's worth of traffic; a group of 16 aligned positions is one 16-byte store a dimension.
// A half warp's worth of consecutive tokens (16) is an item; those that begin a group --
// position a multiple of 16, or the request's first token -- are handled one after another,
// through a tile of shared memory.  Of a group that is not whole, at a request's ends, only the
// request's own bytes are written: the others may be another request's of the same call.  The
// loops are kept short: a version with the group in registers ran 3000 straight instructions,
// which came in from a cold instruction cache at about 10 cycles each.
constexpr int kVKeys = 16;
constexpr int kVPitch = 33;  // 8-byte pieces a row of the tile: its columns on different banks

template <bool E5>
__device__ __forceinline__ void append_v_group(const RopeParams &p, uint2 (&tile)[kVKeys][kVPitch],
                                               uint32_t chunk, int h, int lane)
{
    {
        const int tok = (int)min((uint32_t)p.n, chunk * kVKeys + (lane % kVKeys));
        // ---- this lane's token: its row, and whether it begins a group -------------------
        int64_t row = -1;
        int cnt = 0;
        if (tok < p.n && lane < kVKeys) {
            int lo = 0, hi = p.R;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.cu_tokens + mid) <= tok)
                    lo = mid;
                else
                    hi = mid;
            }
            // (offsets past the tokens there are must not lead past the rows of v)
            const int first = __ldg(p.cu_tokens + lo), last = min(p.n, __ldg(p.cu_tokens + lo + 1));
            const int64_t pos = (int64_t)__ldg(p.start_pos + lo) + (tok - first);
            if (tok >= first && tok < last && pos >= 0 && (pos % kVKeys == 0 || tok == first)) {
                int err = 0;  // flagged with the keys
                row = pool_row(p, __ldg(p.seq_idx + lo), (uint32_t)pos, &err);
                cnt = (int)min((int64_t)(last - tok), kVKeys - pos % kVKeys);
            }
        }
        uint32_t todo = __ballot_sync(0xffffffffu, row >= 0);
        while (todo) {
            const int who = __ffs(todo) - 1;
            todo &= todo - 1;
            const int64_t grow = __shfl_sync(0xffffffffu, row, who);
            const int n = __shfl_sync(0xffffffffu, cnt, who);
            const int gtok = __shfl_sync(0xffffffffu, tok, who);
            const int off = (int)(grow & 63), key0 = off % kVKeys;  // the group's first key there
            const int64_t page = (grow >> 6) + h;
            // ---- key k of the group is token gtok + k - key0: rows to shared memory ----------
            {
                uint2 x[kVKeys];
#pragma unroll
                for (int k = 0; k < kVKeys; ++k) {
                    const int t = k - key0;
                    x[k] = make_uint2(0, 0);
                    if (t >= 0 && t < n)
                        x[k] = __ldcs(reinterpret_cast<const uint2 *>(
                                          p.v + (int64_t)(gtok + t) * p.v_stride + h * 16) + lane);
                }
#pragma unroll
                for (int k = 0; k < kVKeys; ++k)
                    tile[k][lane] = x[k];
            }
            __syncwarp();
            // ---- lanes k and k + 16 take half of key k's magnitudes each ----------------------
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint2 x = tile[lane % kVKeys][lane / kVKeys * 16 + i];
                amax = fmax3(amax, fmaxf(fabsf(bf16_lo(x.x)), fabsf(bf16_hi(x.x))),
                             fmaxf(fabsf(bf16_lo(x.y)), fabsf(bf16_hi(x.y))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
            const float scale = __fdiv_rn(amax, E5 ? 57344.0f : 448.0f);
            uint8_t *const base = reinterpret_cast<uint8_t *>(p.v_dst);
            float *const scales = reinterpret_cast<float *>(base + fp8_codes_bytes(p.num_blocks, p.Hkv));
            if (lane >= key0 && lane < key0 + n)  // lanes 16 .. 31 hold copies
                scales[page * 64 + (off - key0) + lane] = amax > 0.f ? scale : 0.f;
            // ---- codes, a dimension a lane: byte perm16(k) of sixteen is key k's -------------
            const uint16_t *const col = reinterpret_cast<const uint16_t *>(&tile[0][0]) + lane;
            constexpr int kPitch = 4 * kVPitch;  // 16-bit values a row
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                uint32_t word[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    word[w] = 0;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = 2 * w + 8 * e;  // word w: keys 2w, 2w + 1, 2w + 8, 2w + 9
                        const float s0 = __shfl_sync(0xffffffffu, scale, k);
                        const float s1 = __shfl_sync(0xffffffffu, scale, k + 1);
                        const float u = __uint_as_float((uint32_t)col[k * kPitch + 32 * j] << 16);
                        const float v = __uint_as_float((uint32_t)col[(k + 1) * kPitch + 32 * j] << 16);
                        const float a = s0 > 0.f ? __fdiv_rn(u, s0) : 0.f;
                        const float b = s1 > 0.f ? __fdiv_rn(v, s1) : 0.f;
                        word[w] |= (E5 ? f32x2_to_e5m2x2(a, b) : f32x2_to_e4m3x2(a, b)) << (16 * e);
                    }
                }
                uint8_t *const at = base + (page * 128 + 32 * j + lane) * 64 + (off - key0);
                if (n == kVKeys) {
                    *reinterpret_cast<uint4 *>(at) = make_uint4(word[0], word[1], word[2], word[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < kVKeys; ++k)
                        if (k >= key0 && k < key0 + n)
                            at[perm16(k)] = (uint8_t)(word[perm16(k) / 4] >> (8 * (perm16(k) % 4)));
                }
            }
            __syncwarp();
        }
    }
}

// One warp an item: a token and a slice of its head quads (q heads, k heads, then, when
// appending, v heads).  With v_apart the v heads of an FP8 layer are items of their own, ahead
// of the tokens: 16 tokens of a KV head.
template <int KIND, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ uint4 stage_all[KIND == kAppendFp8 ? kWarps * 32 : 1];
    __shared__ uint2 tiles[KIND == kAppendFp8 ? kWarps : 1][kVKeys][kVPitch];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & 7, hl = lane >> 3;
    const bool rot = c < p.rot16;
    const int ca = rot ? c : 2 * c, cb = rot ? c + p.rot16 : 2 * c + 1;
    // this lane computes angles j = 2 hl, 2 hl + 1 of the eight of its chunk pair
    uint64_t F[2] = {0, 0};
    int ax[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int j = 2 * hl + e;
        const int i = INTER ? (j < 4 ? 4 * c + j : 4 * (c + p.rot16) + j - 4) : 8 * c + j;
        if (rot) {
            F[e] = p.turn[i];
            ax[e] = (p.axis2[i >> 4] >> (2 * (i & 15))) & 3;
        }
    }
    const int qq = (p.Hq + 3) >> 2, kq = (p.Hkv + 3) >> 2;
    const int nq = qq + kq + (KIND == kRope || p.v_apart ? 0 : kq);
    const int slices = (nq + p.quads - 1) / p.quads;
    // items count in 32 bits (launch_rope): a 64-bit division an item is 70 instructions
    const uint32_t v_items =
        KIND == kAppendFp8 && p.v_apart ? ((uint32_t)p.n + kVKeys - 1) / kVKeys * p.Hkv : 0;
    const uint32_t items = v_items + (uint32_t)p.n * slices;
    uint8_t *const stage =
        reinterpret_cast<uint8_t *>(stage_all) + (KIND == kAppendFp8 ? (warp * 4 + hl) * 128 : 0);
    grid_dependency_wait();
    for (uint32_t it = blockIdx.x * kWarps + warp; it < items; it += gridDim.x * kWarps) {
        if constexpr (KIND == kAppendFp8) {
            if (it < v_items) {
                if (p.fp8 == 2)
                    append_v_group<true>(p, tiles[warp], it / p.Hkv, it % p.Hkv, lane);
                else
                    append_v_group<false>(p, tiles[warp], it / p.Hkv, it % p.Hkv, lane);
                continue;
            }
        }
        const uint32_t ti = it - v_items;
        const int tok = (int)(ti / slices);
        const int q0 = (int)(ti % slices) * p.quads, q1 = min(nq, q0 + p.quads);
        // head quad qd: q (part 0), k (1) or v (2), its first head h
        uint4 wa[kBatch], wb[kBatch];
        auto load = [&](int qb, bool want_v) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int qd = qb + u;
                const int part = qd < qq ? 0 : (qd < qq + kq ? 1 : 2);
                const int h = 4 * (qd - (part == 0 ? 0 : (part == 1 ? qq : qq + kq))) + hl;
                const uint4 *src = part == 0   ? p.q + (int64_t)tok * p.q_stride
                                   : part == 1 ? p.k + (int64_t)tok * p.k_stride
                                               : p.v + (int64_t)tok * p.v_stride;
                wa[u] = wb[u] = make_uint4(0, 0, 0, 0);
                if (qd < q1 && h < (part == 0 ? p.Hq : p.Hkv) && (part < 2 || want_v)) {
                    wa[u] = __ldcs(src + h * 16 + ca);
                    wb[u] = __ldcs(src + h * 16 + cb);
                }
            }
        };
        load(q0, true);  // ahead of the reads that say where the token belongs
        // ---- the token's request and pool row -------------------------------------
        int64_t row = -1, first_pos = 0;
        bool skip = false;
        if constexpr (KIND != kRope) {
            const int r = find_request(p.cu_tokens, p.R, tok, lane);
            const int first = __ldg(p.cu_tokens + r), last = __ldg(p.cu_tokens + r + 1);
            const int seq = __ldg(p.seq_idx + r);
            first_pos = (int64_t)__ldg(p.start_pos + r) + (tok - first);
            int err = 0;
            if (tok < first || tok >= last || first_pos < 0) {
                err = HSA_DEVERR_BAD_LEN;
                skip = true;
            } else if (!p.ring_mode || tok - first >= (last - first) - p.W) {
                // (an earlier ring token is overwritten later in this same request)
                row = pool_row(p, seq, (uint32_t)first_pos, &err);
            }
            if (err && lane == 0 && q0 == 0)
                set_err(p.dev_err, err);
        }
        if (skip)
            continue;
        // ---- cos and sin of the token's angles ---------------------------------------
        float cs[8], sn[8];
        {
            float c2[2], s2[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t ps = p.pos ? (int64_t)__ldg(p.pos + (int64_t)ax[e] * p.n + tok)
                                         : first_pos;
                const int32_t t = (int32_t)(((uint64_t)ps * F[e]) >> 32);  // 2^-32 of a turn
                sincospif((float)t * 0x1p-31f, &s2[e], &c2[e]);
                c2[e] *= p.scale;
                s2[e] *= p.scale;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cs[j] = __shfl_sync(0xffffffffu, c2[j & 1], (j >> 1) * 8 + c);
                sn[j] = __shfl_sync(0xffffffffu, s2[j & 1], (j >> 1) * 8 + c);
            }
        }
        // ---- the head quads -----------------------------------------------------------
        for (int qb = q0; qb < q1; qb += kBatch) {
            if (qb > q0)
                load(qb, row >= 0);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int qd = qb + u;
                if (qd >= q1)
                    break;
                const int part = qd < qq ? 0 : (qd < qq + kq ? 1 : 2);
                const int h = 4 * (qd - (part == 0 ? 0 : (part == 1 ? qq : qq + kq))) + hl;
                const bool on = h < (part == 0 ? p.Hq : p.Hkv);
                float a[8], b[8];
                if (part < 2) {
                    unpack8(wa[u], a);
                    unpack8(wb[u], b);
                    if (rot) {
                        turn<INTER>(a, b, cs, sn);
                        wa[u] = pack8(a);
                        wb[u] = pack8(b);
                    }
                    uint4 *const dst =
                        part == 0 ? p.q_out + ((int64_t)tok * p.Hq + h) * 16
                                  : (p.k_out ? p.k_out + ((int64_t)tok * p.Hkv + h) * 16 : nullptr);
                    if (on && dst) {
                        __stcs(dst + ca, wa[u]);
                        __stcs(dst + cb, wb[u]);
                    }
                }
                if constexpr (KIND == kAppend) {
                    if (part > 0 && on && row >= 0) {
                        uint4 *const dst = (part == 1 ? p.k_dst : p.v_dst) +
                                           (row + (int64_t)h * (p.ring_mode ? p.W : 64)) * 16;
                        dst[ca] = wa[u];
                        dst[cb] = wb[u];
                    }
                }
                if constexpr (KIND == kAppendFp8) {
                    if (part > 0 && row >= 0) {  // uniform across the warp
                        if (part == 2) {
                            unpack8(wa[u], a);
                            unpack8(wb[u], b);
                        }
                        store_fp8(a, b, ca, cb, on, part == 2, row, on ? h : 0, p, stage, c);
                    }
                }
            }
        }
    }
}

template <int KIND>
cudaError_t launch(const RopeParams &p, unsigned blocks, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.interleaved ? rope_kernel<KIND, true> : rope_kernel<KIND, false>,
                              p);
}

}  // namespace

cudaError_t launch_rope(RopeParams &p, bool append, int sms, cudaStream_t stream)
{
    // An FP8 layer's values by groups of keys, where the requests are long enough to have whole
    // groups and their tokens and heads many enough to fill the SMs.  us by groups, and with a
    // token's values beside its keys:
    //   one request, 2 KV heads: 1500 tokens 18 and 18, 2900 23 and 29; 4 heads: 1024 tokens 20
    //   and 18, 1500 23 and 25, 4096 33 and 45; 8 heads: 700 tokens 21 and 18, 1500 21 and 35
    //   16 requests, 4 heads: 96 tokens each 27 and 25, 128 31 and 27, 256 37 and 43; 8 heads:
    //   64 tokens 29 and 23, 96 31 and 35
    //   64 requests, 4 heads: 32 tokens each 33 and 25, 64 39 and 45
    const int64_t fill = (int64_t)p.n * (p.Hkv + 4);
    p.v_apart = append && p.fp8 && fill >= (p.n >= 300 * (int64_t)p.R ? 12000 : 18000) &&
                p.n >= 32 * (int64_t)p.R && (int64_t)p.n * p.Hkv < (int64_t)1 << 31;
    const int nq = (p.Hq + 3) / 4 + (p.Hkv + 3) / 4 * (append && !p.v_apart ? 2 : 1);
    if (p.n == 0 || nq == 0)
        return cudaSuccess;
    // few tokens: their heads spread over the warps that two blocks an SM have (32 tokens:
    // 2.4 us against 4.0 with a warp a token)
    const int64_t spread = (int64_t)sms * kBlocks * kWarps / p.n;
    p.quads = spread > 1 ? (int32_t)((nq + spread - 1) / spread) : nq;
    const int64_t slices = (nq + p.quads - 1) / p.quads;
    const int64_t v_items = p.v_apart ? ((int64_t)p.n + kVKeys - 1) / kVKeys * p.Hkv : 0;
    int64_t blocks = ((int64_t)p.n * slices + v_items + kWarps - 1) / kWarps;
    blocks = blocks < (int64_t)sms * kBlocks ? blocks : (int64_t)sms * kBlocks;
    if (!append)
        return launch<kRope>(p, (unsigned)blocks, stream);
    return p.fp8 ? launch<kAppendFp8>(p, (unsigned)blocks, stream)
                 : launch<kAppend>(p, (unsigned)blocks, stream);
}

}  // namespace hsa

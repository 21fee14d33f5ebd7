// fd_quant.cuh -- the split kernel's consumer for an 8-bit key/value cache.
//
// Each cached element is a one-byte code, E4M3 (OCP 8-bit floating point:
// sign, 4 exponent bits with bias 7, 3 mantissa bits) or int8, with one
// scale per kv head: k = k_scale[h] * decode(code), v = v_scale[h] *
// decode(code). The "flash decoding论文" page lists INT8/INT4 quantisation
// among PaddleNLP's inference techniques; a cache of one byte per element
// halves the bytes the HBM-bound decode has to stream.
//
// The attention itself is unchanged (fd_split.cuh): per tile, logits, the
// online softmax and the rescaled accumulation of p * v, on tensor cores
// with mma.sync m16n8k16 for every group size (g = 1 included), because
// widening the codes already costs one instruction per two elements and the
// CUDA-core form would add a multiply-add per element on top.
//
//   * Codes are widened to f16 in registers, exactly: every E4M3 value and
//     every int8 value is an f16 value. f16 (not bf16) because the hardware
//     widens E4M3 pairs to f16 pairs in one instruction.
//   * The query is bf16; it enters the contraction as f16 after a per-column
//     power-of-two prescale that puts its largest element in [2^14, 2^15).
//     The prescale is exact, keeps every element inside f16's range, and
//     leaves only elements below 2^-25 of the column's largest rounded; the
//     logit multiplier of each column undoes it together with k_scale and
//     the softmax scale.
//   * Logits, S^T = K Q^T: ldmatrix of the 8-bit tile gives each thread four
//     consecutive codes of one token, which become the A fragment of one
//     16-element k-step once the query's B fragment is loaded in the same
//     order (q[4c .. 4c+3] per thread): the contraction index is only
//     permuted, identically on both sides.
//   * P V, O^T += V^T P^T: V must be transposed (tokens along k). ldmatrix
//     .trans of the 8-bit tile, read as 16-bit elements, hands each thread
//     two tokens x two head dims; one byte permute regroups them into token
//     pairs per head dim before widening. The accumulator rows then hold the
//     even head dims of a chunk (rows 0-7) and the odd ones (rows 8-15),
//     which the store at the end puts back in order.
//   * Softmax with a lazy reference maximum, after FlashDecoding++'s
//     asynchronous softmax with a unified max value (the "flash decoding论文"
//     page names the synchronised partial-softmax update as the problem it
//     removes): each column keeps a reference m and only a tile with a logit
//     above m + kLazy triggers the rescale of the running sum and the
//     accumulators; otherwise its p = 2^(x - m) is summed as is. The result
//     is the same softmax (m cancels in o / l and in the log-sum-exp); the
//     common tile skips the cross-lane max and the accumulator rescale.
//   * P enters as f16 high part + f16 remainder, scaled by 2^kPScale so that
//     small probabilities stay normal f16 numbers; the running sum carries
//     the same factor, so the normalised output is unchanged and only the
//     log-sum-exp is corrected (m - kPScale).
//
// One scale per block of T tokens and kv head (kBlock; T a power of two from
// 16 up, so a scale covers whole 16-token blocks of a warp's slice):
//     x_t = scale log2(e) k_scale[t / T] (q . decode(k_t)),
//     out = sum_t 2^(x_t - m) v_scale[t / T] decode(v_t) / sum_t 2^(x_t - m).
//   * The key scale multiplies the block's logits. The value scale joins the
//     weight: the sum takes p = 2^(x_t - m) and P V takes p r v_scale[t / T],
//     with a power of two r per column, so that the scale enters as a product.
//     r is chosen like m, by the same rare branch, to keep the column's largest
//     contribution p r v_scale in f16's range: P keeps its bits relative to
//     the row's largest contribution, not to its largest scale or weight. r is
//     at most 2^119: a column that has met only zero scales, however heavy,
//     has a finite r, and zero weights times it are zero.
//   * Consumers are what bounds it next to memory (two consumer warps per
//     scheduler; 12 or 16 consumer warps of 16 tokens each were slower, 60 and
//     61 us against 54 on 64 heads over 131072 int8 tokens), so the arithmetic
//     counts: p = 2^(fma(q.k, c, kPScale - m)) and one factor per (block,
//     column) for the values; the test for a new m or r looks at the p and
//     p r v_scale themselves. In short bursts (20 calls a graph, the figures
//     above too), 32 heads over 16384 E4M3 tokens: 27.2 us (one scale per head
//     25.8); 64/8 heads over 131072 int8 tokens: 52.2 us (48.6). Called without
//     a pause the chip's clock falls and the latter takes 56.5 us.
//   * A warp reads its 16-token blocks' scales (through the block table for
//     paged caches) one tile of its group ahead, with loads from L2, so their
//     latency lies behind a tile's arithmetic.
#pragma once

#include "fd_split.cuh"

namespace fd {

template <int D, int NT, bool kE4M3, int kTok = 16, bool kBlock = false, bool kPagedScales = false>
struct QuantConsumer {
    static constexpr int G = 8 * NT;        // columns held (padded)
    static constexpr int kElemBytes = 1;
    static constexpr int kWarpTokens = kTok;          // tokens of each tile per warp (16 or 32)
    static constexpr int MB = kTok / 16;              // 16-token blocks per warp
    static constexpr int KACC = MB == 1 ? 2 : 1;      // logit accumulators per block
    static constexpr bool kInterleaved = false;
    static constexpr bool kTileHook = kBlock;
    static constexpr int KC = D / 16;       // 16-byte chunks of a token = k-steps of S = m-tiles of O^T
    static constexpr int kRowBytes = D;
    // The reference max lags the running max by at most kLazy (base 2), so
    // p = 2^(x - m) <= 2^kLazy; P enters the P V product as p * 2^kPScale,
    // at most 2^15 (f16 tops out near 2^16) and a normal f16 down to p = 2^-21.
    static constexpr float kLazy = 8.f;
    static constexpr float kPScale = 7.f;

    uint32_t qf[NT][KC][2];                 // Q^T as the B operand (f16), per n-tile
    float m[NT][2], l[NT][2];               // reference max (base 2) / partial sum (x 2^kPScale), columns 2c, 2c+1
    float o[NT][KC][4];                     // O^T accumulators (x 2^kPScale, head dims even | odd per chunk)
    int shift[NT][2];                       // causal offset of columns 2c, 2c+1
    float colmul[NT][2];                    // logit multiplier (base 2) of columns 2c, 2c+1
    float kmul, vmul;                       // scale * log2(e) * k_scale[h], and v_scale[h]
    // kBlock only
    float r[NT][2];                         // the power of two in the outputs' weights p r v_scale, columns 2c, 2c+1
    float ks[MB], vs[MB];                   // this tile's key and value scales
    float ks_next[MB], vs_next[MB];         // the group's next tile's scales, on their way
    int page_next[MB];                      // paged: the pages of the tile after that
    const float *kp, *vp;                   // the row's (paged: the head's) scales
    const int32_t *table;                   // paged: the sequence's pages
    int last;                               // the row's last token

    __device__ __forceinline__ void init(const SplitParams &p) {
        const int cc = (threadIdx.x & 31) & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = nt * 8 + 2 * cc + e;
                shift[nt][e] = col < p.cols ? p.q_len - 1 - col / p.g : 0;
            }
    }

    __device__ __forceinline__ void set_row(const SplitParams &p, int h) {
        if constexpr (kBlock) {
            kmul = p.scale_log2e;
            vmul = 1.f;
        } else {
            kmul = p.scale_log2e * __ldg(p.k_scale + h);
            vmul = __ldg(p.v_scale + h);
        }
    }

    // A token of the row (tokens ahead are counted unsigned: a tile or two past a row of nearly 2^31 tokens).
    __device__ __forceinline__ int clip(uint32_t t) const { return static_cast<int>(min(t, static_cast<uint32_t>(last))); }

    // Pages of the slice's 16-token blocks from token t0 on (past the row: of its last token).
    __device__ __forceinline__ void fetch_pages(const SplitParams &p, uint32_t t0) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int t = clip(t0 + 16 * mb);
            page_next[mb] = FD_DCHECK(t >= 0 && (t >> p.page_shift) < p.max_pages) ? __ldcg(table + (t >> p.page_shift)) : -1;
        }
    }

    // Start the loads of the scales of the slice's 16-token blocks from token
    // t0 on. Blocks past the row take its last token's (their weights are 0,
    // and stay 0 times any factor that softmax_block makes of a scale); pages
    // outside the pool read as zeros. L2 loads:
    // the kernel before this one on the stream may have written them after
    // this grid began.
    __device__ __forceinline__ void fetch_scales(const SplitParams &p, uint32_t t0) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            if (mb > 0 && p.blk_shift > 4) continue;   // a slice of 32 tokens is aligned: one scale
            const int t = clip(t0 + 16 * mb);
            if constexpr (kPagedScales) {
                const int page = page_next[mb];
                ks_next[mb] = vs_next[mb] = 0.f;
                if (page < 0 || page >= p.num_pages) continue;
                const size_t at = static_cast<size_t>(page) * p.Hkv * p.blocks +
                                  ((t & ((1 << p.page_shift) - 1)) >> p.blk_shift);
                ks_next[mb] = __ldcg(kp + at);
                vs_next[mb] = __ldcg(vp + at);
            } else {
                const int i = t >> p.blk_shift;
                if (!FD_DCHECK(i >= 0 && i < p.blocks)) continue;
                ks_next[mb] = __ldcg(kp + i);
                vs_next[mb] = __ldcg(vp + i);
            }
        }
    }

    static constexpr uint32_t kStride = kConsumerWarps * kTok;   // tokens from one tile of a group to its next

    // Segment start: the scales of the group's first tile (t0: first token of
    // this warp's slice in it).
    __device__ __forceinline__ void start_segment(const SplitParams &p, const Cursor &c, uint32_t t0, int L) {
        last = L - 1;
        const size_t row = kPagedScales ? static_cast<size_t>(c.h) : static_cast<size_t>(c.b) * p.Hkv + c.h;
        kp = p.k_scale + row * p.blocks;
        vp = p.v_scale + row * p.blocks;
        if constexpr (kPagedScales) {
            table = p.block_table + static_cast<size_t>(c.b) * p.max_pages;
            fetch_pages(p, t0);
            fetch_scales(p, t0);
            fetch_pages(p, t0 + kStride);
        } else {
            fetch_scales(p, t0);
        }
    }

    // Before a tile: its scales have been asked for a tile ago; ask for those
    // of the group's next one.
    __device__ __forceinline__ void before_tile(const SplitParams &p, const Cursor &, uint32_t t0) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {   // (copied here, not where they are asked for: a copy waits for its load)
            const bool first = mb > 0 && p.blk_shift > 4;
            ks[mb] = first ? ks[0] : ks_next[mb];
            vs[mb] = first ? vs[0] : vs_next[mb];
        }
        fetch_scales(p, t0 + kStride);
        if constexpr (kPagedScales) fetch_pages(p, t0 + 2 * kStride);
    }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kBlock ? kNoRef : -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
            if constexpr (kBlock) r[nt][0] = r[nt][1] = 1.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) o[nt][c][0] = o[nt][c][1] = o[nt][c][2] = o[nt][c][3] = 0.f;
        }
    }

    // 16-byte chunk `chunk` of tile row `row`, as TMA's swizzle placed it:
    // 128-byte rows (D = 128) use the 128-byte pattern, 64-byte rows the
    // 64-byte one (chunk bits xor address bits 7..8).
    static __device__ __forceinline__ int swz(int chunk, int row) {
        if constexpr (kRowBytes == 128)
            return chunk ^ (row & 7);
        else
            return chunk ^ ((row >> 1) & 3);
    }

    static __device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
        if constexpr (kE4M3)
            e4m3x4_to_f16(w, lo, hi);
        else
            int8x4_to_f16(w, lo, hi);
    }
    static __device__ __forceinline__ void widen_t(uint32_t w, uint32_t &lo, uint32_t &hi) {
        if constexpr (kE4M3)
            e4m3x4t_to_f16(w, lo, hi);
        else
            int8x4t_to_f16(w, lo, hi);
    }

    // Q^T fragments from the stage's bf16 copy of the row's columns ([cols][D]).
    __device__ __forceinline__ void load_q(const uint8_t *qs, int cols) {
        const int lane = threadIdx.x & 31;
        const int r0 = lane >> 2, cc = lane & 3;
        float cm[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = nt * 8 + r0;
            const bool ok = col < cols;
            const uint2 *qrow = reinterpret_cast<const uint2 *>(qs + (ok ? col : 0) * D * 2);
            float qv[KC][4];
            float mx = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint2 w = qrow[4 * c + cc];   // q[16c + 4cc .. 16c + 4cc + 3]
                qv[c][0] = bf16lo_to_f32(w.x);
                qv[c][1] = bf16hi_to_f32(w.x);
                qv[c][2] = bf16lo_to_f32(w.y);
                qv[c][3] = bf16hi_to_f32(w.y);
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(qv[c][e]));
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));   // the 4 lanes of column r0
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int ex = static_cast<int>((__float_as_uint(mx) >> 23) & 255u);
            const int j = ex == 0 ? 0 : min(141 - ex, 126);          // mx * 2^j in [2^14, 2^15)
            const float up = __uint_as_float(static_cast<uint32_t>(j + 127) << 23);
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                qf[nt][c][0] = ok ? pack_f16x2(qv[c][0] * up, qv[c][1] * up) : 0u;
                qf[nt][c][1] = ok ? pack_f16x2(qv[c][2] * up, qv[c][3] * up) : 0u;
            }
            cm[nt] = kmul * __uint_as_float(static_cast<uint32_t>(127 - j) << 23);   // kmul * 2^-j
        }
        // the softmax needs the multipliers of columns 2cc, 2cc+1, held by lanes 4(2cc+e)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) colmul[nt][e] = __shfl_sync(0xffffffffu, cm[nt], 4 * (2 * cc + e));
    }

    // The slice's value rows from token `valid` on, past the row's end, may
    // hold anything (NaN codes): zero them in the tile, once in a row, rather
    // than test every fragment of every tile. Only this warp reads them; the
    // fence orders the stores before the copy that fills the stage next.
    static __device__ __forceinline__ void clear_rows(uint32_t v_smem, int slice, int valid) {
        const int lane = threadIdx.x & 31;
        const int first = max(valid, 0) * (kRowBytes / 16), end = kWarpTokens * (kRowBytes / 16);
        for (int i = first + lane; i < end; i += 32)   // whole rows: the swizzle only moves chunks inside a row
            st_shared_zero16(v_smem + kWarpTokens * slice * kRowBytes + i * 16);
        fence_proxy_async();
        __syncwarp();
    }

    // This lane's ldmatrix address in a tile at `smem`: row 16 (block) + rr +
    // 8 (mi & 1), chunk mi >> 1, of matrix mi = lane / 8. Chunk pair pc is at
    // that address ^ (pc << 5): the swizzle xors chunk bits with row bits, and
    // tiles are 1024-byte aligned.
    static __device__ __forceinline__ uint32_t lane_addr(uint32_t smem, int slice) {
        const int lane = threadIdx.x & 31, mi = lane >> 3;
        const int row = kWarpTokens * slice + (lane & 7) + 8 * (mi & 1);
        return smem + row * kRowBytes + (swz(mi >> 1, row) << 4);
    }

    // Logits S^T = K Q^T per 16-token block; ldmatrix x4 over two chunks:
    // matrices (tokens 0-7 | 8-15) x (chunk 2pc | 2pc+1). One block keeps
    // two accumulators (even / odd chunks) for two independent mma
    // chains; two blocks already give two.
    __device__ __forceinline__ void logits(uint32_t k_smem, int slice, float (&s)[MB][NT][4]) {
        float s2[MB][NT][4];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mb][nt][e] = s2[mb][nt][e] = 0.f;
        const uint32_t addr = lane_addr(k_smem, slice);
#pragma unroll
        for (int pc = 0; pc < KC / 2; ++pc) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4((addr ^ (pc << 5)) + mb * 16 * kRowBytes, a0, a1, a2, a3);
                uint32_t l0, h0, l1, h1, l2, h2, l3, h3;
                widen(a0, l0, h0);
                widen(a1, l1, h1);
                widen(a2, l2, h2);
                widen(a3, l3, h3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16_16816(s[mb][nt], l0, l1, h0, h1, qf[nt][2 * pc][0], qf[nt][2 * pc][1]);
                    mma_f16_16816(KACC == 2 ? s2[mb][nt] : s[mb][nt], l2, l3, h2, h3, qf[nt][2 * pc + 1][0],
                                  qf[nt][2 * pc + 1][1]);
                }
            }
        }
        if (KACC == 2)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mb][nt][e] += s2[mb][nt][e];
    }

    // P^T fragments of one block and n-tile (f16 high part + remainder).
    static __device__ __forceinline__ void split_p(float p0, float p1, float p2, float p3, uint32_t (&bh)[2],
                                                   uint32_t (&bl)[2]) {
        const uint32_t h01 = pack_f16x2(p0, p1), h23 = pack_f16x2(p2, p3);
        const uint32_t l01 = pack_f16x2(p0 - f16lo_to_f32(h01), p1 - f16hi_to_f32(h01));
        const uint32_t l23 = pack_f16x2(p2 - f16lo_to_f32(h23), p3 - f16hi_to_f32(h23));
        bh[0] = movmatrix_trans(h01);
        bh[1] = movmatrix_trans(h23);
        bl[0] = movmatrix_trans(l01);
        bl[1] = movmatrix_trans(l23);
    }

    // O^T += V^T P^T, one 16-element chunk of head dims per m-tile, one
    // 16-token k-step per block. ldmatrix.trans of the 8-bit tile read as
    // 16-bit elements gives each thread tokens (2cc, 2cc+1) x head dims
    // (2r0, 2r0+1) of a chunk; the widening regroups them into token pairs
    // at head dims 2r0 (accumulator row r0) and 2r0 + 1 (row r0 + 8).
    __device__ __forceinline__ void accumulate(uint32_t v_smem, int slice, const uint32_t (&bh)[MB][NT][2],
                                               const uint32_t (&bl)[MB][NT][2]) {
        const uint32_t addr = lane_addr(v_smem, slice);
        if constexpr (kBlock) {
            // A tile's products are summed from zero and then added to the
            // running sums: the tensor cores' accumulation drops low bits
            // towards zero, a bias that a chain over a run's hundreds of
            // steps adds up (2.1e-6 of the output over 131072 tokens;
            // 6e-7 this way, for one packed addition per two sums and tile).
#pragma unroll
            for (int pc = 0; pc < KC / 2; ++pc) {
                uint32_t a[MB][4];
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
                    ldsm_x4_trans((addr ^ (pc << 5)) + mb * 16 * kRowBytes, a[mb][0], a[mb][1], a[mb][2], a[mb][3]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float t[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) t[nt][0] = t[nt][1] = t[nt][2] = t[nt][3] = 0.f;
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb) {
                        uint32_t A0, A1, A2, A3;
                        widen_t(a[mb][2 * half], A0, A1);
                        widen_t(a[mb][2 * half + 1], A2, A3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16_16816(t[nt], A0, A1, A2, A3, bh[mb][nt][0], bh[mb][nt][1]);
                            mma_f16_16816(t[nt], A0, A1, A2, A3, bl[mb][nt][0], bl[mb][nt][1]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        add2(o[nt][2 * pc + half][0], o[nt][2 * pc + half][1], t[nt][0], t[nt][1]);
                        add2(o[nt][2 * pc + half][2], o[nt][2 * pc + half][3], t[nt][2], t[nt][3]);
                    }
                }
            }
            return;
        }
#pragma unroll
        for (int pc = 0; pc < KC / 2; ++pc) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                uint32_t a[4];
                ldsm_x4_trans((addr ^ (pc << 5)) + mb * 16 * kRowBytes, a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // tokens 0..7 (x) and 8..15 (y) of the block, chunk 2pc + half
                    uint32_t A0, A1, A2, A3;
                    widen_t(a[2 * half], A0, A1);
                    widen_t(a[2 * half + 1], A2, A3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16_16816(o[nt][2 * pc + half], A0, A1, A2, A3, bh[mb][nt][0], bh[mb][nt][1]);
                        mma_f16_16816(o[nt][2 * pc + half], A0, A1, A2, A3, bl[mb][nt][0], bl[mb][nt][1]);
                    }
                }
            }
        }
    }

    // Mask x[mb][nt][..]: token r of block mb is inside column e's causal
    // range when r < valid - 16 mb - shift.
    __device__ __forceinline__ void mask(float (&x)[4], int nt, int vmb) {
        const int r0 = (threadIdx.x & 31) >> 2;
        const int va = vmb - shift[nt][0], vb = vmb - shift[nt][1];
        if (r0 >= va) x[0] = -INFINITY;
        if (r0 >= vb) x[1] = -INFINITY;
        if (r0 + 8 >= va) x[2] = -INFINITY;
        if (r0 + 8 >= vb) x[3] = -INFINITY;
    }

    // One tile: `slice` = this warp's slice of kWarpTokens tokens (MB blocks
    // of 16), `valid` = how many of those tokens are inside the row.
    __device__ __forceinline__ void tile(uint32_t k_smem, uint32_t v_smem, int slice, int valid, float) {
        const bool ends = valid - (FD_MAX_GROUP - 1) < kWarpTokens;   // some column's range may end in this slice
        float s[MB][NT][4];
        uint32_t bh[MB][NT][2], bl[MB][NT][2];
        logits(k_smem, slice, s);
        if constexpr (kBlock)
            softmax_block(s, ends, valid, bh, bl);
        else
            softmax(s, ends, valid, bh, bl);
        if (valid < kWarpTokens) clear_rows(v_smem, slice, valid);
        accumulate(v_smem, slice, bh, bl);
    }

    // Online softmax per column with a lazy reference maximum: m moves
    // (and the accumulators are rescaled) only when a logit of the tile
    // exceeds it by more than kLazy; otherwise p = 2^(x - m) directly.
    // x: the tile's products q . k in, logits out.
    __device__ __forceinline__ void softmax(float (&x)[MB][NT][4], bool ends, int valid, uint32_t (&bh)[MB][NT][2],
                                            uint32_t (&bl)[MB][NT][2]) {
        bool grow = false;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[mb][nt][e] *= colmul[nt][e & 1];
                if (ends) mask(x[mb][nt], nt, valid - 16 * mb);
                const float ta = m[nt][0] + kLazy, tb = m[nt][1] + kLazy;
                grow |= x[mb][nt][0] > ta || x[mb][nt][2] > ta || x[mb][nt][1] > tb || x[mb][nt][3] > tb;
            }
        if (__any_sync(0xffffffffu, grow)) {   // the fallback: a synchronised rescale
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float ma = -INFINITY, mbx = -INFINITY;
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    ma = fmaxf(ma, fmaxf(x[mb][nt][0], x[mb][nt][2]));
                    mbx = fmaxf(mbx, fmaxf(x[mb][nt][1], x[mb][nt][3]));
                }
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) {
                    ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, sh));
                    mbx = fmaxf(mbx, __shfl_xor_sync(0xffffffffu, mbx, sh));
                }
                const float na = fmaxf(m[nt][0], ma), nb = fmaxf(m[nt][1], mbx);
                const float ua = na == -INFINITY ? 0.f : na, ub = nb == -INFINITY ? 0.f : nb;
                const float alpha_a = ex2(m[nt][0] - ua), alpha_b = ex2(m[nt][1] - ub);
                l[nt][0] *= alpha_a;
                l[nt][1] *= alpha_b;
                m[nt][0] = na;
                m[nt][1] = nb;
                rescale(nt, alpha_a, alpha_b);
            }
        }
        // P^T fragments per block, x 2^kPScale
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float ta = kPScale - (m[nt][0] == -INFINITY ? 0.f : m[nt][0]);
            const float tb = kPScale - (m[nt][1] == -INFINITY ? 0.f : m[nt][1]);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                const float p0 = ex2(x[mb][nt][0] + ta), p2 = ex2(x[mb][nt][2] + ta);
                const float p1 = ex2(x[mb][nt][1] + tb), p3 = ex2(x[mb][nt][3] + tb);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                split_p(p0, p1, p2, p3, bh[mb][nt], bl[mb][nt]);
            }
        }
    }

    __device__ __forceinline__ void rescale(int nt, float alpha_a, float alpha_b) {
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            o[nt][c][0] *= alpha_a;
            o[nt][c][1] *= alpha_b;
            o[nt][c][2] *= alpha_a;
            o[nt][c][3] *= alpha_b;
        }
    }

    // The same with one scale per block of tokens: the tile takes
    // p = 2^(x - m + kPScale) into the sum and p f, f = r v_scale, into P V;
    // m and r are right as long as neither p nor p f passes
    // 2^(kLazy + kPScale) (m starts at -3e38, so a first logit gives p = inf).
    // f may pass float's range where the column has contributed next to
    // nothing so far: the test takes it as it is (inf times a p above 0 asks
    // for a new r; inf times 0 is NaN, which fmaxf passes over), P takes it
    // cut to a finite number, so that weight 0 stays 0. After the fallback
    // only weights below 2^-126 of the column's largest can meet the cut.
    // m is a whole number, so that r and the references' differences are
    // exact. s: the tile's products q . k.
    static constexpr float kNoRef = -3e38f;
    static constexpr float kMaxLog2R = 119.f;     // an output of 2^-126 then still has P at 1, a normal f16
    static constexpr float kMinLog2R = -126.f;    // a scale of nearly 2^128 then has P below 2^10
    static constexpr float kMaxF = 8.507059e37f;  // 2^126
    // 2^e of whole e in [-126, 126], and back.
    static __device__ __forceinline__ float exp2i(float e) {
        return __uint_as_float(static_cast<uint32_t>(static_cast<int>(e) + 127) << 23);
    }
    static __device__ __forceinline__ float log2i(float x) {
        return static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 127);
    }
    __device__ __forceinline__ void softmax_block(float (&s)[MB][NT][4], bool ends, int valid,
                                                  uint32_t (&bh)[MB][NT][2], uint32_t (&bl)[MB][NT][2]) {
        constexpr float kMost = 32768.f;   // 2^(kLazy + kPScale)
        static_assert(kLazy + kPScale == 15.f && kPScale == 7.f, "kMost, and the factor that to_smem takes off");
        float p[MB][NT][4], f[MB][NT][2];
        float most = 0.f;
        auto weights = [&] {
            most = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float ta = kPScale - m[nt][0], tb = kPScale - m[nt][1];
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    const float ca = colmul[nt][0] * ks[mb], cb = colmul[nt][1] * ks[mb];
                    fma2(s[mb][nt][0], s[mb][nt][1], ca, cb, ta, tb, p[mb][nt][0], p[mb][nt][1]);
                    fma2(s[mb][nt][2], s[mb][nt][3], ca, cb, ta, tb, p[mb][nt][2], p[mb][nt][3]);
                    if (ends) mask(p[mb][nt], nt, valid - 16 * mb);
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[mb][nt][e] = ex2(p[mb][nt][e]);
                    const float fa = r[nt][0] * vs[mb], fb = r[nt][1] * vs[mb];
                    const float ma = fmaxf(p[mb][nt][0], p[mb][nt][2]), mbx = fmaxf(p[mb][nt][1], p[mb][nt][3]);
                    most = fmaxf(fmaxf(most, ma), mbx);
                    most = fmaxf(fmaxf(most, ma * fa), mbx * fb);
                    f[mb][nt][0] = fminf(fa, kMaxF);
                    f[mb][nt][1] = fminf(fb, kMaxF);
                }
            }
        };
        weights();
        if (__any_sync(0xffffffffu, most > kMost)) {   // the fallback: a synchronised rescale of sum and outputs
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float xm = kNoRef, ym = kNoRef;   // the column's largest logit, and largest log2 of a contribution
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb) {
                        const float c = colmul[nt][e] * ks[mb];
                        float z[4] = {s[mb][nt][0] * c, s[mb][nt][1] * c, s[mb][nt][2] * c, s[mb][nt][3] * c};
                        if (ends) mask(z, nt, valid - 16 * mb);
                        const float x = fmaxf(z[e], z[e + 2]);
                        xm = fmaxf(xm, x);
                        ym = fmaxf(ym, x + lg2(vs[mb]));
                    }
#pragma unroll
                    for (int sh = 4; sh < 32; sh <<= 1) {
                        xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, sh));
                        ym = fmaxf(ym, __shfl_xor_sync(0xffffffffu, ym, sh));
                    }
                    xm = fmaxf(m[nt][e], ceilf(xm));
                    const float dm = m[nt][e] - xm;
                    // relative to the new m: the largest contribution that r stood for so far, and the tile's
                    const float was = dm - log2i(r[nt][e]);
                    const float y = fminf(fmaxf(fmaxf(ceilf(ym - xm), was), -kMaxLog2R), -kMinLog2R);
                    const float alpha = ex2(was - y);
                    l[nt][e] *= ex2(dm);
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        o[nt][c][e] *= alpha;
                        o[nt][c][e + 2] *= alpha;
                    }
                    m[nt][e] = xm;
                    r[nt][e] = exp2i(-y);
                }
            weights();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                l[nt][0] += p[mb][nt][0] + p[mb][nt][2];
                l[nt][1] += p[mb][nt][1] + p[mb][nt][3];
                split_p(p[mb][nt][0] * f[mb][nt][0], p[mb][nt][1] * f[mb][nt][1], p[mb][nt][2] * f[mb][nt][0],
                        p[mb][nt][3] * f[mb][nt][1], bh[mb][nt], bl[mb][nt]);
            }
    }

    // This warp's (o, m, l) into a merge buffer slot: o[G][D] with the head
    // dims back in order and the value scale applied, then m[G] (base 2, with
    // the 2^kPScale factor of o and l taken off), l[G].
    __device__ __forceinline__ void to_smem(float *wb) {
        constexpr int S = merge_head_stride<D>();
        const int lane = threadIdx.x & 31;
        const int r0 = lane >> 2, cc = lane & 3;
        const int dlo = 2 * r0;   // head dim of accumulator row r0 within its chunk (row r0 + 8: dlo + 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], sh);
            const int ha = nt * 8 + 2 * cc, hb = ha + 1;
            float va = vmul, vb = vmul;
            if constexpr (kBlock) {
                // without r and 2^kPScale (taken off the sum, not off m: the hardware log2's error grows with
                // the sum's distance from 1), and the merge's "no token" for a column without
                va = exp2i(-log2i(r[nt][0]) - kPScale);
                vb = exp2i(-log2i(r[nt][1]) - kPScale);
                l[nt][0] *= 1.f / 128.f;
                l[nt][1] *= 1.f / 128.f;
                if (m[nt][0] == kNoRef) m[nt][0] = -INFINITY;
                if (m[nt][1] == kNoRef) m[nt][1] = -INFINITY;
            }
            // dims d0 and d0 + 1 of one head as one 8-byte store; with the padded
            // head stride the 16 lanes of each half warp fill all 32 banks
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int d0 = 16 * c + dlo;
                *reinterpret_cast<float2 *>(wb + ha * S + d0) = make_float2(o[nt][c][0] * va, o[nt][c][2] * va);
                *reinterpret_cast<float2 *>(wb + hb * S + d0) = make_float2(o[nt][c][1] * vb, o[nt][c][3] * vb);
            }
            if (r0 == 0) {
                constexpr float off = kBlock ? 0.f : kPScale;
                wb[G * S + ha] = m[nt][0] == -INFINITY ? -INFINITY : m[nt][0] - off;
                wb[G * S + hb] = m[nt][1] == -INFINITY ? -INFINITY : m[nt][1] - off;
                wb[G * S + G + ha] = l[nt][0];
                wb[G * S + G + hb] = l[nt][1];
            }
        }
    }
};

}  // namespace fd

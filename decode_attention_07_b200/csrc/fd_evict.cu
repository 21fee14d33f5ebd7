// fd_evict.cu -- fd_evict: cut a cache to a budget by accumulated attention
// weight, in two kernels.
//
// Mathematics. For a row (sequence b, kv head h) of L tokens with totals w:
//   L <= keep: every token stays. Otherwise the last `recent` tokens stay and,
//   of the M = L - recent others, the k = keep - recent with the largest w
//   (ties to the lowest index; NaN below everything). Kept tokens stay in
//   order, so the newest ones are still the last ones.
// Selection is a radix select on an unsigned key that orders as w does: four
// passes over 8 bits from the top, each a histogram of the keys that match the
// digits found so far, give the k-th largest key; a token is kept if its key
// is above it, or equal and among the first equal ones. The counts are
// integers, so nothing depends on the order of the atomics.
//
// Select kernel: a cluster of 1 to 8 blocks per row, each with a contiguous
// slice of its tokens; a pass exchanges 256 bins over distributed shared
// memory. Totals crowd into few digits (a few binades, many zeros), so a
// histogram has 8 columns that lanes take by turns: at most 4 additions of a
// warp meet. Up to 16 keys a thread stay in registers over all passes; longer
// slices read their totals again from L2.
// Gather kernel: 16-byte vectors, 64 kept tokens a block, all of a thread's
// loads in flight before its first store.
//
// What bounds it: the kept keys and values, read once and written once
// (8 D bytes a token); selection reads 4 bytes a cached token and comes
// before the first copy can start. 8 rows of 131072 tokens cut to 32768
// (275 MB): 64 us, of which the copy 42 (6.4 TB/s, a copy's rate) and the
// selection 20 (2.6 a pass, 0.8 of it the cluster barrier); 512 rows of up to
// 4096 cut to 1000 (474 MB): 89 us. Slices past the registers (rows of more than
// 131072 tokens, or fewer blocks a row) are read again in each pass: 8 rows of
// 262144 cut to 65536 take 130 us, 32 rows of 131072 cut to 32768 211, and one
// row of a million cut to 100000, which eight blocks select, 159. Clusters of 16 blocks (of 512 threads)
// were no faster: their barrier and remote reads grow as their slices shrink.
#include <cooperative_groups.h>

#include "fd_host.cuh"

namespace fd {

namespace cg = cooperative_groups;

constexpr int kKeys = 16;                                   // keys a thread of the select kernel holds
constexpr int kShortSlice = 256 * kKeys;                    // slices that 256 threads hold
constexpr int kBins = 256;
constexpr int kCols = 8;                                    // histogram columns: lanes 8 apart share one
constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 64;

struct EvictParams {
    const uint16_t *k, *v;           // [B, Hkv, Lmax, D]
    const float *w;                  // [B, Hkv, Lmax]
    const int32_t *seqlens;          // [B]
    uint16_t *k_out, *v_out;         // [B, Hkv, out_len, D]
    float *w_out;                    // [B, Hkv, out_len]
    int32_t *kept;                   // [B, Hkv, keep]
    int32_t *seqlens_out;            // [B]
    int B, Hkv, Lmax, keep, recent, out_len;
};

// Unsigned order of totals: NaN first (1), then -inf .. +inf, -0 as +0. 0
// is below them all and stands for "no token" in a batch's last part.
__device__ __forceinline__ uint32_t order_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    const uint32_t k = static_cast<int32_t>(u) < 0 ? ~u : u | 0x80000000u;
    return w != w ? 1u : k;
}

// Sum of the words of histogram row `bin`, which it clears.
__device__ __forceinline__ uint32_t take_row(uint32_t *hist, int bin) {
    uint4 *row = reinterpret_cast<uint4 *>(hist + bin * kCols);
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < kCols / 4; ++j) {
        const uint4 v = row[j];
        row[j] = make_uint4(0, 0, 0, 0);
        sum += (v.x + v.y) + (v.z + v.w);
    }
    return sum;
}

// kT threads: 256 for slices of up to 4096 tokens (more rows at once on an
// SM), 1024 for longer ones.
template <int kT>
__global__ void __launch_bounds__(kT) fd_select_kernel(const EvictParams p) {
    constexpr int kWarps = kT / 32;
    constexpr int kBatch = kT * kKeys;           // tokens of one batch of a slice
    constexpr int kCounts = kKeys * kWarps;
    __shared__ __align__(16) uint32_t hist[kBins * kCols];   // this block's histogram
    __shared__ uint32_t bins[2][kBins];          // its sums, by turns: the cluster reads one while the next is made
    __shared__ uint32_t counts[kCounts];         // a batch's (above | equal << 16) by step and warp
    __shared__ uint32_t warp_sums[kWarps];
    __shared__ uint32_t found[3];                // digit, keys above it, keys in it
    __shared__ uint32_t slice_sums[2];           // kept-above and equal keys of this block's slice

    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependents_launch();
    for (int i = tid; i < kBins * kCols / 4; i += kT) reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0, 0, 0, 0);
    const long long u = blockIdx.x / C;
    const int b = static_cast<int>(u / p.Hkv), h = static_cast<int>(u - static_cast<long long>(b) * p.Hkv);
    grid_dependency_wait();
    const int L = clamp_len(__ldcg(p.seqlens + b), p.Lmax);
    int32_t *kept = p.kept + static_cast<size_t>(u) * p.keep;
    const int n = min(L, p.keep);
    if (h == 0 && rank == 0 && tid == 0) p.seqlens_out[b] = n;
    const int step = C * kT, me = rank * kT + tid;
    if (L <= p.keep) {   // the same in every block of the cluster: nothing to select
        for (long long i = me; i < p.keep; i += step) kept[i] = i < L ? static_cast<int>(i) : -1;
        return;
    }
    const int M = L - p.recent, k = p.keep - p.recent;
    for (long long i = me; i < p.recent; i += step) kept[k + i] = static_cast<int>(M + i);
    if (k == 0) return;

    // this block's slice [lo, hi) of the candidates
    const long long slice = (static_cast<long long>(M) + C - 1) / C;
    const long long lo = min(rank * slice, static_cast<long long>(M)), hi = min(lo + slice, static_cast<long long>(M));
    const float *w = p.w + static_cast<size_t>(u) * p.Lmax;
    const bool resident = slice <= kBatch;
    uint32_t key[kKeys];
    // the batch's keys, thread-striped (token base + i * kT + tid)
    auto load = [&](long long base) {
        const int n_left = static_cast<int>(min(hi - base, static_cast<long long>(kBatch))) - tid;
        const float *at = w + base + tid;
        float x[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) x[i] = i * kT < n_left ? __ldcg(at + i * kT) : 0.f;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) key[i] = i * kT < n_left ? order_key(x[i]) : 0u;
    };
    if (resident) load(lo);
    __syncthreads();   // hist is clear

    uint32_t prefix = 0, need = static_cast<uint32_t>(k);
    int shift = 32;           // the key's bits from `shift` up are settled: they are prefix's
    bool whole_bin = false;   // every key that matches the prefix is kept
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        constexpr int kDigit = 8;
        if (whole_bin) break;
        const int down = 24 - kDigit * pass;
        for (long long base = lo; base < hi; base += kBatch) {
            if (!resident) load(base);
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
                if (pass == 0 || (key[i] >> (down + (pass == 0 ? 0 : kDigit))) == (prefix >> (down + (pass == 0 ? 0 : kDigit))))
                    atomicAdd(&hist[((key[i] >> down) & 255u) * kCols + (lane & (kCols - 1))], 1u);
        }
        __syncthreads();
        // the digit whose bin holds the need-th key of the cluster from the
        // top: thread i takes bin 255 - i, which it sums and clears. Another
        // block's bins of this pass are whole after the cluster barrier, and
        // written again two passes on, after the next one.
        uint32_t c = 0, incl = 0;
        const int bin = kBins - 1 - tid;
        if (tid < kBins) c = take_row(hist, bin);
        if (C > 1) {
            uint32_t *mine = bins[pass & 1];
            if (tid < kBins) mine[bin] = c;
            cluster.sync();
            if (tid < kBins) {
                uint32_t others[8];   // all remote reads on their way at once (C <= 8)
#pragma unroll
                for (int r = 0; r < 8; ++r) others[r] = r < C ? cluster.map_shared_rank(mine, r)[bin] : 0u;
                c = 0;
#pragma unroll
                for (int r = 0; r < 8; ++r) c += others[r];
            }
        }
        if (tid < kBins) {
            incl = c;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, s);
                if (lane >= s) incl += y;
            }
            if (lane == 31) warp_sums[warp] = incl;
        }
        __syncthreads();
        if (tid < kBins) {
            uint32_t before = incl - c;
#pragma unroll
            for (int i = 0; i < kBins / 32; ++i) before += i < warp ? warp_sums[i] : 0u;
            if (before < need && before + c >= need) {
                found[0] = static_cast<uint32_t>(bin);
                found[1] = before;
                found[2] = c;
            }
        }
        __syncthreads();
        prefix |= found[0] << down;
        shift = down;
        need -= found[1];
        whole_bin = found[2] == need;
        // (found is written again only after the next pass's barriers)
    }
    // kept: keys above `top`, and the first `need` of those from `prefix` to `top`
    const uint32_t top = prefix | ((1u << shift) - 1u);

    // The batch's counts of both kinds by step and warp become exclusive sums
    // in token order (packed above | equal << 16: at most 16384 of each kind).
    // Returns the batch's total.
    auto rank_batch = [&]() -> uint32_t {
        uint32_t n_mine = 0;   // lane i: step i's counts
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const uint32_t ng = __popc(__ballot_sync(0xffffffffu, key[i] > top));
            const uint32_t ne = __popc(__ballot_sync(0xffffffffu, key[i] >= prefix)) - ng;
            if (lane == i) n_mine = ng | (ne << 16);
        }
        __syncthreads();   // the last batch's sums have been read
        if (lane < kKeys) counts[lane * kWarps + warp] = n_mine;
        __syncthreads();
        uint32_t c = 0, incl = 0;
        if (tid < kCounts) {
            c = counts[tid];
            incl = c;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, s);
                if (lane >= s) incl += y;
            }
            if (lane == 31) warp_sums[warp] = incl;
        }
        __syncthreads();
        uint32_t total = 0, before = incl - c;
#pragma unroll
        for (int i = 0; i < kCounts / 32; ++i) {
            const uint32_t x = warp_sums[i];
            before += i < warp ? x : 0u;
            total += x;
        }
        if (tid < kCounts) counts[tid] = before;
        __syncthreads();
        return total;
    };
    static_assert(kKeys <= 32 && kCounts <= kT && kCounts % 32 == 0, "one scan of the counts");
    static_assert(kBatch < 65536, "packed counts");

    uint32_t gt_before = 0, eq_before = 0, total = 0;
    if (C > 1) {   // this slice's counts, then those of the slices before it
        uint32_t gt = 0, eq = 0;
        for (long long base = lo; base < hi; base += kBatch) {
            if (!resident) load(base);
            total = rank_batch();
            gt += total & 0xffffu;
            eq += total >> 16;
        }
        if (tid == 0) {
            slice_sums[0] = gt;
            slice_sums[1] = eq;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            gt_before += cluster.map_shared_rank(slice_sums, r)[0];
            eq_before += cluster.map_shared_rank(slice_sums, r)[1];
        }
        cluster.barrier_arrive();   // this thread reads no other block's memory from here on
    }
    const unsigned lower = (1u << lane) - 1u;
    for (long long base = lo; base < hi; base += kBatch) {
        if (!resident) load(base);
        if (C == 1 || !resident) total = rank_batch();   // (one batch: still there)
        const int t_mine = static_cast<int>(base) + tid;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const bool g = key[i] > top, ge = key[i] >= prefix;
            const unsigned bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, ge) & ~bg;
            if ((bg | be) == 0) continue;
            const uint32_t before = counts[i * kWarps + warp];
            const uint32_t gb = gt_before + (before & 0xffffu) + __popc(bg & lower);
            const uint32_t eb = eq_before + (before >> 16) + __popc(be & lower);
            if (g || (ge && eb < need)) kept[gb + min(eb, need)] = t_mine + i * kT;
        }
        gt_before += total & 0xffffu;
        eq_before += total >> 16;
    }
    if (C > 1) cluster.barrier_wait();   // no block leaves while another reads its shared memory
}

template <int D>
__global__ void __launch_bounds__(kGatherThreads) fd_gather_kernel(const EvictParams p, long long chunks, long long total) {
    constexpr int kVec = D / 8;                                     // 16-byte vectors of a token
    constexpr int NI = kGatherTokens * kVec / kGatherThreads;       // vectors per thread, of K and of V
    constexpr int kRows = kGatherThreads / kVec;
    __shared__ int idx[kGatherTokens];
    grid_dependents_launch();
    grid_dependency_wait();
    const int tid = threadIdx.x, row0 = tid / kVec, col = (tid % kVec) * 8;
    for (long long item = blockIdx.x; item < total; item += gridDim.x) {
        const long long u = item / chunks;
        const int s0 = static_cast<int>((item - u * chunks) * kGatherTokens);
        __syncthreads();   // the last item's positions have been read
        if (tid < kGatherTokens) {
            const int s = s0 + tid;
            const int t = s < p.keep ? __ldcg(p.kept + static_cast<size_t>(u) * p.keep + s) : -1;
            idx[tid] = t;
            if (s < p.out_len)
                p.w_out[static_cast<size_t>(u) * p.out_len + s] =
                    t >= 0 ? __ldcg(p.w + static_cast<size_t>(u) * p.Lmax + t) : 0.f;
        }
        __syncthreads();
        if (idx[0] < 0) continue;   // kept positions come first
        const uint16_t *k = p.k + static_cast<size_t>(u) * p.Lmax * D + col;
        const uint16_t *v = p.v + static_cast<size_t>(u) * p.Lmax * D + col;
        uint4 x[NI], y[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int t = idx[row0 + i * kRows];
            if (t >= 0) {
                const size_t at = static_cast<size_t>(t) * D;
                x[i] = __ldcs(reinterpret_cast<const uint4 *>(k + at));
                y[i] = __ldcs(reinterpret_cast<const uint4 *>(v + at));
            }
        }
        const size_t out = (static_cast<size_t>(u) * p.out_len + s0) * D + col;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int r = row0 + i * kRows;
            if (idx[r] >= 0) {
                *reinterpret_cast<uint4 *>(p.k_out + out + static_cast<size_t>(r) * D) = x[i];
                *reinterpret_cast<uint4 *>(p.v_out + out + static_cast<size_t>(r) * D) = y[i];
            }
        }
    }
}

}  // namespace fd


extern "C" {

int fd_evict(int B, int Hkv, int D, int max_len, int keep, int recent, int out_len, const uint16_t *k_cache,
             const uint16_t *v_cache, const float *weights, const int32_t *seqlens, uint16_t *k_out, uint16_t *v_out,
             float *weights_out, int32_t *kept, int32_t *seqlens_out, void *stream) {
    using namespace fdh;
    int rc = check_shape(B, Hkv, Hkv, D, max_len);
    if (rc != FD_OK) return rc;
    if (keep < 1 || recent < 0 || recent > keep || out_len < keep) return FD_ERR_SHAPE;
    if (!seqlens || !k_out || !v_out || !weights_out || !kept || !seqlens_out) return FD_ERR_NULL_POINTER;
    if (max_len > 0 && (!k_cache || !v_cache || !weights)) return FD_ERR_NULL_POINTER;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return FD_ERR_ALIGNMENT;
    if (!aligned(weights, 4) || !aligned(weights_out, 4) || !aligned(kept, 4) || !aligned(seqlens, 4) ||
        !aligned(seqlens_out, 4))
        return FD_ERR_ALIGNMENT;
    // the blocks copy in no order: what is written may not be what another still reads
    const size_t rows = static_cast<size_t>(B) * Hkv;
    const size_t in_b = rows * max_len * D * 2, out_b = rows * out_len * D * 2;
    const size_t win_b = rows * max_len * 4, wout_b = rows * out_len * 4, kept_b = rows * keep * 4;
    const size_t len_b = static_cast<size_t>(B) * 4;
    const void *ins[4] = {k_cache, v_cache, weights, seqlens};
    const size_t in_n[4] = {in_b, in_b, win_b, len_b};
    const void *outs[5] = {k_out, v_out, weights_out, kept, seqlens_out};
    const size_t out_n[5] = {out_b, out_b, wout_b, kept_b, len_b};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 4; ++j)
            if (overlap(outs[i], out_n[i], ins[j], in_n[j])) return FD_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], out_n[i], outs[j], out_n[j])) return FD_ERR_OVERLAP;
    }
    if (rows * 8 > 0x7fffffffULL) return FD_ERR_SHAPE;   // grid x of the select kernel
    int sms;
    if ((rc = device_sms(&sms)) != FD_OK) return rc;

    fd::EvictParams p;
    p.k = k_cache;
    p.v = v_cache;
    p.w = weights;
    p.seqlens = seqlens;
    p.k_out = k_out;
    p.v_out = v_out;
    p.w_out = weights_out;
    p.kept = kept;
    p.seqlens_out = seqlens_out;
    p.B = B;
    p.Hkv = Hkv;
    p.Lmax = max_len;
    p.keep = keep;
    p.recent = recent;
    p.out_len = out_len;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // blocks per row: more while a slice is longer than 4096 tokens and the
    // rows leave SMs idle; 8 at most (clusters of 16 of these blocks fit the
    // device 7 at a time, one fewer than the rows of a long single sequence)
    int C = 1;
    while (C < 8 && max_len / C > fd::kShortSlice && static_cast<long long>(rows) * C * 2 <= sms) C *= 2;
    const dim3 blocks(static_cast<unsigned>(rows * C));
    rc = max_len <= static_cast<long long>(fd::kShortSlice) * C
             ? launch_dependent(fd::fd_select_kernel<256>, blocks, 256, 0, st, C, p)
             : launch_dependent(fd::fd_select_kernel<1024>, blocks, 1024, 0, st, C, p);
    if (rc != FD_OK) return rc;
    const long long chunks = (static_cast<long long>(out_len) + fd::kGatherTokens - 1) / fd::kGatherTokens;
    const long long total = static_cast<long long>(rows) * chunks;
    const dim3 grid(static_cast<unsigned>(total < 0x7fffffffLL ? total : 0x7fffffffLL));
    return D == 128 ? launch_dependent(fd::fd_gather_kernel<128>, grid, fd::kGatherThreads, 0, st, 1, p, chunks, total)
                    : launch_dependent(fd::fd_gather_kernel<64>, grid, fd::kGatherThreads, 0, st, 1, p, chunks, total);
}

}  // extern "C"

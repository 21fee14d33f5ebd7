// fd_weights.cu -- fd_decode_weights: decode attention that also adds each
// cached token's attention weight to a running total.
//
//     w_out[b, h, t] = w_in[b, h, t] + sum over the columns c of kv head h of
//                      exp(z_{c,t} - lse_c)                      (t < seqlens[b])
//
// A weight needs its row's final log-sum-exp, known only once every split has
// been merged. So the split kernel (its consumers' kLogits form) also stores
// each logit, 4 bytes per (token, column) beside the 4 D bytes of K and V it
// reads, and one pass after it turns them into weights: reading K again
// instead would move 2 D bytes per token. The logits go [row][token][column]:
// a warp of the grouped consumer stores whole 32-byte sectors, and the pass
// reads a token's columns as one vector.
//
// What bounds it: 4 D bytes of K and V and 8 bytes of totals per (token, kv
// head); the logits' round trip is 8 bytes a column, mostly through L2. One
// sequence of 16384 tokens, 32 heads (273 MB): 46 us, 5.9 TB/s (attention
// alone 41); 131072 tokens, 64 / 8 heads (545 MB): 96 us in short bursts (80),
// 98 sustained; the second kernel adds a launch and two dependent loads, 4 to
// 6 us, which is most of a small call.
#include "fd_host.cuh"

namespace fd {

constexpr int kWeightsThreads = 256;
// Tokens of one row per block: all of a thread's loads fit its registers at
// once (512 tokens of 16 columns: window of queries 25.2 -> 23.7 us).
__host__ __device__ constexpr int weights_tokens(int lcols) { return lcols > 8 ? 512 : 1024; }

struct WeightsParams {
    const float *logits;      // [B, Hkv, Lmax, lcols], base 2
    const float *lse;         // [B, q_len, Hq], natural log
    const float *w_in;        // [B, Hkv, Lmax] or NULL (zeros)
    float *w_out;             // [B, Hkv, Lmax]; may be w_in
    const int32_t *seqlens;
    int B, q_len, Hq, Hkv, g, Lmax, cols, lcols;
};

// kVec floats.
template <int kVec>
__device__ __forceinline__ void load_logits(const float *at, float (&x)[kVec]) {
    if constexpr (kVec == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(at));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else if constexpr (kVec == 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(at));
        x[0] = v.x, x[1] = v.y;
    } else {
        x[0] = __ldcg(at);
    }
}

// Base-2 log-sum-exp of column col of row (b, h); +inf where the column saw
// nothing and for padding columns, whose weights 2^(x - inf) are then 0.
__device__ __forceinline__ float column_lse2(const WeightsParams &p, int b, int h, int col) {
    if (col >= p.cols) return INFINITY;
    const int j = col / p.g, i = col - j * p.g;
    const float ls = __ldcg(p.lse + (static_cast<size_t>(b) * p.q_len + j) * p.Hq + h * p.g + i);
    return ls == -INFINITY ? INFINITY : ls * kLog2eF;
}

// A token's logits are kN vectors of kVec floats (kVec * kN = lcols). A warp
// takes 32 tokens at a time, read as 32 kN consecutive vectors, one per lane
// and load; where kN is a power of two the kN lanes of a token add up their
// parts and each lane ends with one token of the 32. (Other kN: a token per
// lane.) All of a step's loads are on their way before the first is used
// (between seqlens and the buffers' end they read the unused part). The
// log-sum-exps are read by one warp per block: every block of a row wants the
// same 64 bytes, and asking for them from every warp kept one L2 slice busy
// for 7 us of 15 on a row of 131072 tokens. Logits are read for the last
// time here, so the whole lines of them leave L2 without being written to
// memory (33 MB a call at 64 heads over 131072 tokens: 107 -> 101 us).
template <int kVec, int kN>
__global__ void __launch_bounds__(kWeightsThreads) fd_weights_kernel(const WeightsParams p) {
    constexpr bool kSplit = (kN & (kN - 1)) == 0;
    constexpr int kTokens = weights_tokens(kVec * kN);
    constexpr int kSteps = kTokens / kWeightsThreads;             // 32-token steps of a warp
    __shared__ float lse2_of[FD_MAX_GROUP];
    grid_dependents_launch();
    grid_dependency_wait();
    const int u = blockIdx.x, b = u / p.Hkv, h = u - b * p.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int L = clamp_len(__ldcg(p.seqlens + b), p.Lmax);
    if (static_cast<long long>(blockIdx.y) * kTokens >= L) return;
    float column = 0.f;
    if (threadIdx.x < FD_MAX_GROUP) column = column_lse2(p, b, h, threadIdx.x);
    bool have_lse2 = false;
    const int part = kSplit ? lane % kN : 0;
    float lse2[kSplit ? kVec : kVec * kN];
    const size_t row = static_cast<size_t>(u) * p.Lmax;
    // the lane's token among a step's 32
    const int mine = kSplit ? part * (32 / kN) + lane / kN : lane;
    for (long long t0 = static_cast<long long>(blockIdx.y) * kTokens; t0 < L;
         t0 += static_cast<long long>(gridDim.y) * kTokens) {
        float x[kSteps][kN][kVec], w[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const long long t = t0 + s * kWeightsThreads + warp * 32;
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const int tok = kSplit ? (j * 32 + lane) / kN : lane;
                const int off = kSplit ? (j * 32 + lane) * kVec : (lane * kN + j) * kVec;
                if (t + tok < p.Lmax)
                    load_logits<kVec>(p.logits + (row + t) * (kVec * kN) + off, x[s][j]);
                else
#pragma unroll
                    for (int k = 0; k < kVec; ++k) x[s][j][k] = -INFINITY;
            }
            w[s] = p.w_in && t + mine < p.Lmax ? __ldcg(p.w_in + row + t + mine) : 0.f;
        }
        if (!have_lse2) {   // once, with the first step's loads on their way
            if (threadIdx.x < FD_MAX_GROUP) lse2_of[threadIdx.x] = column;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < (kSplit ? kVec : kVec * kN); ++k) lse2[k] = lse2_of[part * kVec + k];
            have_lse2 = true;
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const long long t = t0 + s * kWeightsThreads + warp * 32;
            float sum = 0.f;
            if constexpr (kSplit) {
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    float v = 0.f;
#pragma unroll
                    for (int k = 0; k < kVec; ++k) v += ex2(x[s][j][k] - lse2[k]);
#pragma unroll
                    for (int sh = 1; sh < kN; sh <<= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
                    sum = j == part ? v : sum;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kN; ++j)
#pragma unroll
                    for (int k = 0; k < kVec; ++k) sum += ex2(x[s][j][k] - lse2[j * kVec + k]);
            }
            if (t + mine < L) p.w_out[row + t + mine] = w[s] + sum;
            __syncwarp();   // every lane has its logits
            const float *lines = p.logits + (row + t) * (kVec * kN);
            if (lane < kVec * kN && t + 32 <= p.Lmax && (reinterpret_cast<uintptr_t>(lines) & 127) == 0)
                discard_l2_128(lines + lane * 32);
        }
    }
}

}  // namespace fd

namespace fdh {

int take_weights_error(int *word) { return take_error_word(fd::g_fd_error_word, word); }

namespace {

size_t logits_bytes(int B, int Hkv, int max_len, int cols) {
    return static_cast<size_t>(B) * Hkv * static_cast<size_t>(max_len) * fd::logit_cols(cols) * sizeof(float);
}

// The workspace: the logits, then the split kernel's own (both 256-byte aligned).
size_t split_offset(int B, int Hkv, int max_len, int cols) { return align256(logits_bytes(B, Hkv, max_len, cols)); }

int launch_logits(int D, bool rows_map, const CUtensorMap &tk, const CUtensorMap &tv, const fd::SplitParams &p,
                  cudaStream_t st) {
    if (D == 128) {
        if (rows_map) return launch_split_t<128, fd::HeadConsumer<128, true, 16, true>, true, false>(tk, tv, p, st);
        if (p.cols <= 8) return launch_split_t<128, fd::GroupConsumer<128, 1, false, true>, true, false>(tk, tv, p, st);
        return launch_split_t<128, fd::GroupConsumer<128, 2, false, true>, true, false>(tk, tv, p, st);
    }
    if (p.cols == 1) return launch_split_t<64, fd::HeadConsumer<64, false, 16, true>, true, false>(tk, tv, p, st);
    if (p.cols <= 8) return launch_split_t<64, fd::GroupConsumer<64, 1, false, true>, true, false>(tk, tv, p, st);
    return launch_split_t<64, fd::GroupConsumer<64, 2, false, true>, true, false>(tk, tv, p, st);
}

template <int kVec, int kN>
int launch_weights(dim3 grid, const fd::WeightsParams &w, cudaStream_t st) {
    return launch_dependent(fd::fd_weights_kernel<kVec, kN>, grid, fd::kWeightsThreads, 0, st, 1, w);
}

int check_weights_shape(int B, int q_len, int Hq, int Hkv, int D, int max_len) {
    if (q_len < 1 || q_len > FD_MAX_GROUP) return FD_ERR_SHAPE;
    const int rc = check_shape(B, Hq, Hkv, D, max_len);
    if (rc != FD_OK) return rc;
    return static_cast<long long>(Hq) * q_len / Hkv > FD_MAX_GROUP ? FD_ERR_GROUP : FD_OK;
}

}  // namespace
}  // namespace fdh

extern "C" {

size_t fd_weights_workspace_bytes(int B, int q_len, int Hq, int Hkv, int D, int max_len, int num_splits) {
    if (fdh::check_weights_shape(B, q_len, Hq, Hkv, D, max_len) != FD_OK) return 0;
    if (num_splits < 1 || num_splits > FD_MAX_SPLITS) return 0;
    return fdh::split_offset(B, Hkv, max_len, Hq / Hkv * q_len) +
           fdh::workspace_bytes(B, Hq * q_len, Hkv, D, num_splits);
}

int fd_decode_weights(int B, int q_len, int Hq, int Hkv, int D, int max_len, const uint16_t *q,
                      const uint16_t *k_cache, const uint16_t *v_cache, const int32_t *seqlens, float scale, float *out,
                      float *lse, const float *weights_in, float *weights_out, void *workspace, size_t workspace_bytes,
                      int num_splits, void *stream) {
    using namespace fdh;
    int rc = check_weights_shape(B, q_len, Hq, Hkv, D, max_len);
    if (rc != FD_OK) return rc;
    if (num_splits < 0) return FD_ERR_SPLITS;
    if (max_len > 0) {
        if (!weights_out) return FD_ERR_NULL_POINTER;
        if (!aligned(weights_out, 4) || (weights_in && !aligned(weights_in, 4))) return FD_ERR_ALIGNMENT;
        // in place, or apart: a total may not be another's input
        const size_t n = static_cast<size_t>(B) * Hkv * max_len * sizeof(float);
        if (weights_in && weights_in != weights_out && overlap(weights_in, n, weights_out, n)) return FD_ERR_OVERLAP;
    }
    int S = num_splits;
    // the argument checks that need no plan, then the plan, then the workspace for it
    Problem pr = make_problem(B, Hq * q_len, Hkv, D, max_len, q, k_cache, v_cache, seqlens, scale, out, lse, nullptr, 0,
                              1, stream);
    if ((rc = check_problem(pr, true)) != FD_OK) return rc;
    if (S == 0 && (S = fd_plan(B, Hq, Hkv, D, max_len)) < 0) return S;
    const int cols = Hq / Hkv * q_len;
    const size_t head = split_offset(B, Hkv, max_len, cols);
    if (head > 0) {
        if (!workspace || workspace_bytes < head) return FD_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return FD_ERR_ALIGNMENT;
    }
    pr.num_splits = S;
    pr.ws = workspace ? static_cast<char *>(workspace) + head : nullptr;
    pr.ws_bytes = workspace ? workspace_bytes - head : 0;
    if ((rc = check_problem(pr, true)) != FD_OK) return rc;
    pr.Hq = Hq;
    int sms;
    if ((rc = device_sms(&sms)) != FD_OK) return rc;
    {   // what is written may not be what the kernels still read, nor one another
        const size_t cache = static_cast<size_t>(B) * Hkv * max_len * D * 2, totals = cache / D * 2;
        const size_t rows = static_cast<size_t>(B) * q_len * Hq;
        const void *ins[4] = {q, k_cache, v_cache, seqlens};
        const size_t in_n[4] = {rows * D * 2, cache, cache, static_cast<size_t>(B) * 4};
        const void *outs[4] = {out, lse, workspace, weights_out};
        const size_t out_n[4] = {rows * D * 4, rows * 4,
                                 workspace ? head + fdh::workspace_bytes(B, Hq * q_len, Hkv, D, S) : 0, totals};
        for (int i = 0; i < 4; ++i) {
            for (int j = 0; j < 4; ++j)
                if (overlap(outs[i], out_n[i], ins[j], in_n[j])) return FD_ERR_OVERLAP;
            for (int j = 0; j < i; ++j)
                if (overlap(outs[i], out_n[i], outs[j], out_n[j])) return FD_ERR_OVERLAP;
            if (i < 3 && weights_in && overlap(outs[i], out_n[i], weights_in, totals)) return FD_ERR_OVERLAP;
        }
    }

    CUtensorMap tk, tv;
    std::memset(&tk, 0, sizeof tk);
    std::memset(&tv, 0, sizeof tv);
    const long long rows = static_cast<long long>(B) * Hkv;
    const bool rows_map = D == 128 && cols == 1;   // one copy per K or V tile (see encode_cache_map_rows)
    if (max_len > 0) {
        if (rows_map) {
            if ((rc = encode_cache_map_rows(&tk, k_cache, max_len, rows)) != FD_OK) return rc;
            if ((rc = encode_cache_map_rows(&tv, v_cache, max_len, rows)) != FD_OK) return rc;
        } else {
            if ((rc = encode_cache_map(&tk, k_cache, D, max_len, rows)) != FD_OK) return rc;
            if ((rc = encode_cache_map(&tv, v_cache, D, max_len, rows)) != FD_OK) return rc;
        }
    }
    fd::SplitParams p = split_params(pr, q_len, nullptr);
    p.logits = static_cast<float *>(workspace);
    if ((rc = launch_logits(D, rows_map, tk, tv, p, pr.stream)) != FD_OK) return rc;
    if (max_len == 0) return FD_OK;   // no token anywhere

    fd::WeightsParams w;
    w.logits = p.logits;
    w.lse = lse;
    w.w_in = weights_in;
    w.w_out = weights_out;
    w.seqlens = seqlens;
    w.B = B;
    w.q_len = q_len;
    w.Hq = Hq;
    w.Hkv = Hkv;
    w.g = p.g;
    w.Lmax = max_len;
    w.cols = cols;
    w.lcols = fd::logit_cols(cols);
    const int per = fd::weights_tokens(w.lcols);
    const long long chunks = (static_cast<long long>(max_len) + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(chunks < 65535 ? chunks : 65535));
    switch (w.lcols) {
        case 1: return launch_weights<1, 1>(grid, w, pr.stream);
        case 2: return launch_weights<2, 1>(grid, w, pr.stream);
        case 4: return launch_weights<4, 1>(grid, w, pr.stream);
        case 6: return launch_weights<2, 3>(grid, w, pr.stream);
        case 8: return launch_weights<4, 2>(grid, w, pr.stream);
        case 10: return launch_weights<2, 5>(grid, w, pr.stream);
        case 12: return launch_weights<4, 3>(grid, w, pr.stream);
        case 14: return launch_weights<2, 7>(grid, w, pr.stream);
        default: return launch_weights<4, 4>(grid, w, pr.stream);
    }
}

}  // extern "C"

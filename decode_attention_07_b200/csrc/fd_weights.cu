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
// head); the logits' round trip is 8 bytes a column, mostly through L2.
#include "fd_host.cuh"

namespace fd {

constexpr int kWeightsThreads = 256;
constexpr int kWeightsTokens = 1024;   // tokens of one row per block

struct WeightsParams {
    const float *logits;      // [B, Hkv, Lmax, lcols], base 2
    const float *lse;         // [B, q_len, Hq], natural log
    const float *w_in;        // [B, Hkv, Lmax] or NULL (zeros)
    float *w_out;             // [B, Hkv, Lmax]; may be w_in
    const int32_t *seqlens;
    int B, q_len, Hq, Hkv, g, Lmax, cols, lcols;
};

// kVec floats of a token's logits per load; lcols is a multiple of kVec.
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

template <int kVec>
__global__ void __launch_bounds__(kWeightsThreads) fd_weights_kernel(const WeightsParams p) {
    __shared__ float lse2[FD_MAX_GROUP];   // base-2 log-sum-exp of the row's columns; columns that saw nothing: +inf
    grid_dependents_launch();
    grid_dependency_wait();
    const int u = blockIdx.x, b = u / p.Hkv, h = u - b * p.Hkv;
    const int L = clamp_len(__ldcg(p.seqlens + b), p.Lmax);
    if (static_cast<long long>(blockIdx.y) * kWeightsTokens >= L) return;
    if (threadIdx.x < FD_MAX_GROUP) {
        const int col = threadIdx.x;
        float v = INFINITY;                // 2^(x - inf) = 0: padding columns too
        if (col < p.cols) {
            const int j = col / p.g, i = col - j * p.g;
            const float ls = __ldcg(p.lse + (static_cast<size_t>(b) * p.q_len + j) * p.Hq + h * p.g + i);
            if (ls != -INFINITY) v = ls * kLog2eF;
        }
        lse2[col] = v;
    }
    __syncthreads();
    const size_t row = static_cast<size_t>(u) * p.Lmax;
    for (long long t0 = static_cast<long long>(blockIdx.y) * kWeightsTokens; t0 < L;
         t0 += static_cast<long long>(gridDim.y) * kWeightsTokens) {
#pragma unroll
        for (int i = 0; i < kWeightsTokens / kWeightsThreads; ++i) {
            const long long t = t0 + i * kWeightsThreads + threadIdx.x;
            if (t >= L) break;
            const size_t at = row + static_cast<size_t>(t);
            float w = p.w_in ? __ldcg(p.w_in + at) : 0.f;
            float sum = 0.f;
            for (int c = 0; c < p.lcols; c += kVec) {
                float x[kVec];
                load_logits<kVec>(p.logits + at * p.lcols + c, x);
#pragma unroll
                for (int k = 0; k < kVec; ++k) sum += ex2(x[k] - lse2[c + k]);
            }
            p.w_out[at] = w + sum;
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
    const long long chunks = (static_cast<long long>(max_len) + fd::kWeightsTokens - 1) / fd::kWeightsTokens;
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(chunks < 65535 ? chunks : 65535));
    if (w.lcols % 4 == 0) return launch_dependent(fd::fd_weights_kernel<4>, grid, fd::kWeightsThreads, 0, pr.stream, 1, w);
    if (w.lcols % 2 == 0) return launch_dependent(fd::fd_weights_kernel<2>, grid, fd::kWeightsThreads, 0, pr.stream, 1, w);
    return launch_dependent(fd::fd_weights_kernel<1>, grid, fd::kWeightsThreads, 0, pr.stream, 1, w);
}

}  // extern "C"

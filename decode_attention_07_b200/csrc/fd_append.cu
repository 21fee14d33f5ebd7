// fd_append.cu -- fd_quant_append and fd_quant_append_paged: new bf16 tokens
// into an 8-bit cache with one scale per block of T tokens and kv head.
//
// Mathematics, per (sequence, kv head, touched block) and for K and V apart,
// with a = the largest magnitude among the block's new tokens and R the
// largest code (448 for E4M3, 127 for int8):
//     s_new = a / R rounded up to 8 significant bits (a bf16 number),
//     s     = s_new, or max(s_old, s_new) when the block holds older tokens,
//     code  = round(x / s) half to even; older codes, only when s > s_old:
//             round(decode(code) * s_old / s).
// Why 8 significant bits: then x (8 bits) against t * s for a rounding
// boundary t (at most 8 bits) compares integers of at most 16 bits, so a
// quotient is either exactly on the boundary or at least 2^-17 (relative) off
// it. A quotient good to 2^-22 that is exact whenever x / s is representable
// therefore rounds as the real quotient does: codes are the definition's, bit
// for bit, without a division per element. Older codes, a rare
// path, and scales with more bits (a caller's own) or tiny ones go through 64
// bits: the codes are the definition's for those too.
// The quotient: q0 = x r with r = 1/s to nearest, then one correction step
// q = q0 + (x - q0 s) r with fused multiply-adds. If x / s = t is
// representable, q0 = t (1 + d) with |d| < 2^-22, the residual x - q0 s =
// -t d s is exact, and q is t up to a relative 2^-45, which rounds to t.
//
// What bounds it: 4 D bytes read and 2 D written per (token, kv head); for a
// token or two, the launch and two dependent loads (length, then data).
// 16384 tokens of 32 heads (403 MB): 68 us in short bursts (5.9 TB/s), 75 us
// sustained; 16 uneven chunks of 1000 tokens into pages (72 MB): 15.9 us; one
// token for each of 64 sequences: 5.3 us in bursts, 5.8 sustained. Wider groups (4 loads a thread) and
// several blocks of tokens in turn per thread block measured slower: what
// counts is loads in flight, 8 a thread at 1024 threads a SM.
// A group of 1 to 8 warps per (block of tokens, kv head, K or V), 8 loads of
// 16 bytes in flight a thread: the new tokens stay in registers between the
// maximum and the rounding, so they are read once. 256 threads a block: the
// groups of neighbouring heads, whose tokens lie side by side in a
// token-major source.
#include "fd_host.cuh"

namespace fd {

constexpr int kAppendThreads = 256;

struct AppendParams {
    const uint16_t *src[2];          // k_new, v_new
    uint8_t *codes[2];               // k, v codes (contiguous cache or pool)
    float *scale[2];
    long long stride_b, stride_t, stride_h;   // elements between sequences, tokens, heads of k_new / v_new
    const int32_t *new_lens;         // [B] or NULL: n_new
    const int32_t *seqlens;          // [B], the new tokens included
    int B, n_new, Hkv, max_len;
    int touched;                     // blocks of tokens a run of n_new tokens can touch
    int blocks;                      // scale blocks per row, or per page
    const int32_t *block_table;      // paged only
    int max_pages, page_shift, num_pages, nhd;
};

// a / R rounded up to 8 significant bits: up to a float, then up on the
// float's bits, of which 16 go in the normal range and all but the leading 8
// below it (a is at least 2^-133, so a / R still has 8 there).
template <bool kE4M3>
__device__ __forceinline__ float block_scale(float a) {
    const uint32_t u = __float_as_uint(__fdiv_ru(a, kE4M3 ? 448.f : 127.f));
    const int drop = min(16, max(0, 24 - __clz(u)));
    return __uint_as_float((u + (1u << drop) - 1u) >> drop << drop);
}

// A 64-bit quotient as a float that rounds on as it would: towards zero, the
// last bit set where that dropped anything (so it never lands on a rounding
// boundary of the codes by accident).
__device__ __forceinline__ float to_odd(double d) {
    const float f = __double2float_rz(d);
    return static_cast<double>(f) == d ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// The comment's quotient holds for this scale: 8 significant bits (a caller's
// own older scale may have more), and neither its reciprocal nor the residual
// leaves float's normal range.
__device__ __forceinline__ bool fast_scale(float s) {
    return (__float_as_uint(s) & 0xffffu) == 0 && s >= 8.6736174e-19f;   // 2^-60
}
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q0 = x * r;
    return fmaf(fmaf(-q0, s, x), r, q0);
}

// Four quotients to four codes (byte 0 = the first), half to even. The int8
// codes of |y| <= 127: adding 1.5 * 2^23 leaves the integer in the low bits.
template <bool kE4M3>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (kE4M3) {
        uint32_t w;
        asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
            : "=r"(w)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return w;
    } else {
        const float k = 12582912.f;
        const uint32_t ab = __byte_perm(__float_as_uint(a + k), __float_as_uint(b + k), 0x0040);
        const uint32_t cd = __byte_perm(__float_as_uint(c + k), __float_as_uint(d + k), 0x0040);
        return __byte_perm(ab, cd, 0x5410);
    }
}

// Four codes to their values.
template <bool kE4M3>
__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
    uint32_t lo, hi;
    if constexpr (kE4M3)
        e4m3x4_to_f16(w, lo, hi);
    else
        int8x4_to_f16(w, lo, hi);
    v[0] = f16lo_to_f32(lo);
    v[1] = f16hi_to_f32(lo);
    v[2] = f16lo_to_f32(hi);
    v[3] = f16hi_to_f32(hi);
}

// Eight bf16 values at `at` to codes, for any scale.
template <bool kE4M3>
__device__ __noinline__ uint2 encode_exactly(const uint16_t *at, float s) {
    uint32_t w[2];
    for (int e = 0; e < 2; ++e) {
        const uint32_t w0 = reinterpret_cast<const uint32_t *>(at)[2 * e];
        const uint32_t w1 = reinterpret_cast<const uint32_t *>(at)[2 * e + 1];
        float v[4] = {bf16lo_to_f32(w0), bf16hi_to_f32(w0), bf16lo_to_f32(w1), bf16hi_to_f32(w1)};
        for (int k = 0; k < 4; ++k) v[k] = s > 0.f ? to_odd(static_cast<double>(v[k]) / static_cast<double>(s)) : 0.f;
        w[e] = encode4<kE4M3>(v[0], v[1], v[2], v[3]);
    }
    return make_uint2(w[0], w[1]);
}

// Eight codes at `at` from scale s_old to the larger s.
template <bool kE4M3>
__device__ __noinline__ void recode(uint8_t *at, float s_old, float s) {
    const uint2 old = __ldcg(reinterpret_cast<const uint2 *>(at));
    uint32_t w[2] = {old.x, old.y};
    for (int e = 0; e < 2; ++e) {
        float v[4];
        decode4<kE4M3>(w[e], v);
        for (int k = 0; k < 4; ++k) {
            v[k] = to_odd(static_cast<double>(v[k]) * s_old / static_cast<double>(s));
            if (!kE4M3) v[k] = fminf(fmaxf(v[k], -127.f), 127.f);   // the code -128 is not written
        }
        w[e] = encode4<kE4M3>(v[0], v[1], v[2], v[3]);
    }
    *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
}

// Threads per (block of tokens, head): 8 chunks of 16 bytes each.
template <int D, int T>
__host__ __device__ constexpr int append_group() {
    return T * D / 64 < 32 ? 32 : T * D / 64;
}

template <int D, int T, bool kE4M3, bool kPaged>
__global__ void __launch_bounds__(kAppendThreads, 4) fd_append_kernel(const AppendParams p) {
    constexpr int kVec = D / 8;                       // 16-byte chunks of a token
    constexpr int kGroup = append_group<D, T>();      // threads of a group
    constexpr int kGroups = kAppendThreads / kGroup;  // heads of a block
    constexpr int NI = T * kVec / kGroup;             // chunks per thread
    constexpr int kRows = kGroup / kVec;              // tokens per step
    __shared__ float warp_max[kAppendThreads / 32];
    grid_dependents_launch();
    grid_dependency_wait();
    const int tid = threadIdx.x % kGroup, group = threadIdx.x / kGroup;
    const int h = (blockIdx.x >> 1) * kGroups + group, kv = blockIdx.x & 1;
    if (h >= p.Hkv) return;
    const int row0 = tid / kVec, col = (tid % kVec) * 8;
    for (long long b = blockIdx.z; b < p.B; b += gridDim.z) {
        const long long end = __ldcg(p.seqlens + b);
        const int count = p.new_lens ? min(max(__ldcg(p.new_lens + b), 0), p.n_new) : p.n_new;
        const long long start = end - count;
        const int lo = static_cast<int>(start > 0 ? start : 0);   // lo <= hi's type: seqlens and max_len are int32
        const int hi = static_cast<int>(end < p.max_len ? end : p.max_len);
        for (long long j = blockIdx.y; j < p.touched; j += gridDim.y) {
            const long long t0l = (static_cast<long long>(lo / T) + j) * T;
            if (t0l >= hi || lo >= hi) break;
            const int t0 = static_cast<int>(t0l);
            // the block's new tokens, in registers (asked for before anything
            // else is waited for), and their largest magnitude
            uint4 x[NI];
            const uint16_t *src = p.src[kv] + b * p.stride_b + h * p.stride_h + col;
            __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
            const uint16_t *at = src + (t0 + row0 - start) * p.stride_t;
            const long long step = kRows * p.stride_t;
            const int first = lo - t0 - row0, past = hi - t0 - row0;   // new: i * kRows in [first, past)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (i * kRows >= first && i * kRows < past) x[i] = __ldcs(reinterpret_cast<const uint4 *>(at));
                at += step;
            }
            // where the block's codes and scale are
            uint8_t *codes = p.codes[kv];
            size_t scale_at, row_stride = D;
            if constexpr (kPaged) {
                const int page = __ldcg(p.block_table + b * p.max_pages + (t0 >> p.page_shift));
                if (page < 0 || page >= p.num_pages) continue;    // outside the pool: dropped
                const int off = t0 & ((1 << p.page_shift) - 1);
                if (p.nhd) {
                    row_stride = static_cast<size_t>(p.Hkv) * D;
                    codes += (((static_cast<size_t>(page) << p.page_shift) + off) * p.Hkv + h) * D;
                } else {
                    codes += (((static_cast<size_t>(page) * p.Hkv + h) << p.page_shift) + off) * D;
                }
                scale_at = (static_cast<size_t>(page) * p.Hkv + h) * p.blocks + off / T;
            } else {
                const size_t u = static_cast<size_t>(b) * p.Hkv + h;
                codes += (u * p.max_len + t0) * D;
                scale_at = u * p.blocks + t0 / T;
            }
            const bool has_old = t0 < lo;
            const float s_old = has_old ? __ldcg(p.scale[kv] + scale_at) : 0.f;

#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e])));
            }
            float a = fmaxf(__low2float(m2), __high2float(m2));
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, sh));
            if constexpr (kGroup > 32) {   // over the group's warps
                float *wm = warp_max + group * (kGroup / 32);
                named_barrier_sync(1 + group, kGroup);   // the last maxima have been read
                if ((tid & 31) == 0) wm[tid >> 5] = a;
                named_barrier_sync(1 + group, kGroup);
#pragma unroll
                for (int w = 0; w < kGroup / 32; ++w) a = fmaxf(a, wm[w]);
            }

            const float s = fmaxf(block_scale<kE4M3>(a), s_old);
            if (tid == 0 && !(has_old && s == s_old)) p.scale[kv][scale_at] = s;
            if (fast_scale(s)) {
                const float rs = __frcp_rn(s);
                uint8_t *to = codes + row0 * row_stride + col;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const uint2 c = make_uint2(
                        encode4<kE4M3>(quotient(bf16lo_to_f32(x[i].x), s, rs), quotient(bf16hi_to_f32(x[i].x), s, rs),
                                       quotient(bf16lo_to_f32(x[i].y), s, rs), quotient(bf16hi_to_f32(x[i].y), s, rs)),
                        encode4<kE4M3>(quotient(bf16lo_to_f32(x[i].z), s, rs), quotient(bf16hi_to_f32(x[i].z), s, rs),
                                       quotient(bf16lo_to_f32(x[i].w), s, rs), quotient(bf16hi_to_f32(x[i].w), s, rs)));
                    if (i * kRows >= first && i * kRows < past) *reinterpret_cast<uint2 *>(to) = c;
                    to += kRows * row_stride;
                }
            } else {   // any other scale: 64-bit quotients, the tokens read again
#pragma unroll 1
                for (int r = row0; r < T; r += kRows)
                    if (t0 + r >= lo && t0 + r < hi)
                        *reinterpret_cast<uint2 *>(codes + r * row_stride + col) =
                            encode_exactly<kE4M3>(src + (t0 + r - start) * p.stride_t, s);
            }
            if (has_old && s > s_old) {   // the scale grew: the older codes follow (rare: about log T times a block)
#pragma unroll 1
                for (int r = row0; t0 + r < lo; r += kRows)
                    recode<kE4M3>(codes + r * row_stride + col, s_old, s);
            }
        }
    }
}

}  // namespace fd

namespace fdh {
namespace {

template <int D, int T, bool kE4M3>
int launch_append(const fd::AppendParams &p, cudaStream_t st) {
    constexpr int heads = fd::kAppendThreads / fd::append_group<D, T>();
    const dim3 grid(static_cast<unsigned>((p.Hkv + heads - 1) / heads) * 2u, static_cast<unsigned>(p.touched < 65535 ? p.touched : 65535),
                    static_cast<unsigned>(p.B < 65535 ? p.B : 65535));
    return p.block_table ? launch_dependent(fd::fd_append_kernel<D, T, kE4M3, true>, grid, fd::kAppendThreads, 0, st, 1, p)
                         : launch_dependent(fd::fd_append_kernel<D, T, kE4M3, false>, grid, fd::kAppendThreads, 0, st, 1,
                                            p);
}

template <int D, bool kE4M3>
int launch_append_t(int T, const fd::AppendParams &p, cudaStream_t st) {
    switch (T) {
        case 16: return launch_append<D, 16, kE4M3>(p, st);
        case 32: return launch_append<D, 32, kE4M3>(p, st);
        case 64: return launch_append<D, 64, kE4M3>(p, st);
        default: return launch_append<D, 128, kE4M3>(p, st);
    }
}

int append(int B, int n_new, int Hkv, int D, int max_len, int block_tokens, int kv_type, const uint16_t *k_new,
           const uint16_t *v_new, long long stride_b, long long stride_t, long long stride_h, const int32_t *new_lens,
           const int32_t *seqlens, uint8_t *k, uint8_t *v, float *k_scale, float *v_scale, void *stream,
           const PagedLayout *pl) {
    if (n_new < 0) return FD_ERR_SHAPE;
    if (kv_type != FD_KV_E4M3 && kv_type != FD_KV_INT8) return FD_ERR_SHAPE;
    if (!valid_block(block_tokens) || (pl && block_tokens > pl->page_size)) return FD_ERR_SHAPE;
    int rc = check_shape(B, Hkv, Hkv, D, max_len);
    if (rc != FD_OK) return rc;
    if (Hkv > 0x3fffffff) return FD_ERR_SHAPE;   // grid x = 2 Hkv
    if (n_new == 0 || max_len == 0) return FD_OK;
    if (!k_new || !v_new || !seqlens || !k || !v || !k_scale || !v_scale) return FD_ERR_NULL_POINTER;
    if (pl && !pl->block_table) return FD_ERR_NULL_POINTER;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k, 16) || !aligned(v, 16)) return FD_ERR_ALIGNMENT;
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(seqlens, 4)) return FD_ERR_ALIGNMENT;
    if (new_lens && !aligned(new_lens, 4)) return FD_ERR_ALIGNMENT;
    if (pl && !aligned(pl->block_table, 4)) return FD_ERR_ALIGNMENT;
    // rows of 16-byte vectors
    if (stride_b % 8 != 0 || stride_t % 8 != 0 || stride_h % 8 != 0) return FD_ERR_ALIGNMENT;
    int sms;
    if ((rc = device_sms(&sms)) != FD_OK) return rc;
    fd::AppendParams p;
    std::memset(&p, 0, sizeof p);
    p.src[0] = k_new;
    p.src[1] = v_new;
    p.codes[0] = k;
    p.codes[1] = v;
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.stride_b = stride_b;
    p.stride_t = stride_t;
    p.stride_h = stride_h;
    p.new_lens = new_lens;
    p.seqlens = seqlens;
    p.B = B;
    p.n_new = n_new;
    p.Hkv = Hkv;
    p.max_len = max_len;
    p.touched = static_cast<int>((static_cast<long long>(n_new) + block_tokens - 2) / block_tokens + 1);
    p.blocks = static_cast<int>(((pl ? pl->page_size : max_len) + block_tokens - 1LL) / block_tokens);
    if (pl) {
        p.block_table = pl->block_table;
        p.max_pages = pl->max_pages;
        while ((1 << p.page_shift) < pl->page_size) ++p.page_shift;
        p.num_pages = pl->num_pages;
        p.nhd = pl->nhd ? 1 : 0;
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (D == 128)
        return kv_type == FD_KV_E4M3 ? launch_append_t<128, true>(block_tokens, p, st)
                                     : launch_append_t<128, false>(block_tokens, p, st);
    return kv_type == FD_KV_E4M3 ? launch_append_t<64, true>(block_tokens, p, st)
                                 : launch_append_t<64, false>(block_tokens, p, st);
}

}  // namespace
}  // namespace fdh

extern "C" {

int fd_quant_append(int B, int n_new, int Hkv, int D, int max_len, int block_tokens, int kv_type,
                    const uint16_t *k_new, const uint16_t *v_new, long long stride_b, long long stride_t,
                    long long stride_h, const int32_t *new_lens, const int32_t *seqlens, uint8_t *k_codes,
                    uint8_t *v_codes, float *k_scale, float *v_scale, void *stream) {
    return fdh::append(B, n_new, Hkv, D, max_len, block_tokens, kv_type, k_new, v_new, stride_b, stride_t, stride_h,
                       new_lens, seqlens, k_codes, v_codes, k_scale, v_scale, stream, nullptr);
}

int fd_quant_append_paged(int B, int n_new, int Hkv, int D, int page_size, int num_pages, int max_pages_per_seq,
                          int kv_layout, int block_tokens, int kv_type, const uint16_t *k_new, const uint16_t *v_new,
                          long long stride_b, long long stride_t, long long stride_h, const int32_t *new_lens,
                          const int32_t *block_table, const int32_t *seqlens, uint8_t *k_pages, uint8_t *v_pages,
                          float *k_scale, float *v_scale, void *stream) {
    long long max_len = 0;
    const int rc = fdh::check_paged(page_size, num_pages, max_pages_per_seq, kv_layout, &max_len);
    if (rc != FD_OK) return rc;
    const fdh::PagedLayout pl{block_table, page_size, num_pages, max_pages_per_seq, kv_layout == FD_KV_NHD};
    return fdh::append(B, n_new, Hkv, D, static_cast<int>(max_len), block_tokens, kv_type, k_new, v_new, stride_b,
                       stride_t, stride_h, new_lens, seqlens, k_pages, v_pages, k_scale, v_scale, stream, &pl);
}

}  // extern "C"

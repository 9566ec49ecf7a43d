// The prompt pass: the gated Delta recurrence (and plain decayed linear
// attention) over many tokens of each request of a plan.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "stepq_serve.cuh"

namespace stepq {
namespace {

constexpr unsigned kFull = 0xffffffffu;

template <class T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// ---------------------------------------------------------------------------
// Token by token.  A CTA holds 32 value columns of one state in registers (16
// values a thread: 4 key rows x 4 columns) and takes the request's tokens in
// turn.  Columns are independent, so four CTAs share a state.  With p = S'^T k
// and r = S'^T q summed in the same pass, u = beta (v - p) and out = r + (k.q) u:
// one exchange between the warps a token.  A single token is bound by the
// state's bytes (64 KiB in, 64 KiB out a head): five CTAs an SM keep enough of
// them under way, and the states pass the caches (nothing reads them again).
// Single tokens, gated Delta rule, bf16, 64 requests of 32 heads (270 MB): 53 us,
// 5.1 TB/s; a gate per key row, fp32, 128 of 32 (547 MB): 105 us, 5.2 TB/s; plain,
// binary16, 256 of 32 (1.08 GB): 183 us, 5.9 TB/s, of 6.5 that a copy reaches.
// Every further token costs its chain of loads, shuffles and one barrier: 1.6 us
// where all CTAs lie on the GPU at once, 45 us a token for 128 requests of 32.
// ---------------------------------------------------------------------------
constexpr int kStepCols = 32;
constexpr int kStepThreads = 256;
constexpr int kStepSlices = kDV / kStepCols;

template <class T, int V>
__global__ void __launch_bounds__(kStepThreads, 5) k_prompt_steps(PromptArgs a)
{
    // three buffers: the one written while token t is processed was last read
    // by token t - 2, which every thread has left at the barrier of t - 1
    __shared__ float sk[3][kDK], sq[3][kDK], sa[3][kDK], sv[3][kStepCols];
    __shared__ __align__(16) float red[2][8][2 * kStepCols];
    __shared__ float red_kq[2][8];
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
    const int slice = blockIdx.x % kStepSlices;
    const int item = blockIdx.x / kStepSlices, r = item / a.heads, h = item - r * a.heads;
    // one wait for all of the request's entries
    const int live = a.p.live[r], t0 = a.p.starts[r], t1 = a.p.starts[r + 1];
    const bool fresh = a.p.fresh[r] != 0;
    if (live < 0) return;
    const int c = tid & 7, g = tid >> 3;  // columns 4c .. 4c+3 of the slice, key rows g + 32 i
    const int hq = h / a.share;
    float *Sp = a.S + ((long long)(a.by_slot ? live : r) * a.heads + h) * (kDK * kDV) + slice * kStepCols + 4 * c;
    const T *qg = static_cast<const T *>(a.q), *kg = static_cast<const T *>(a.k), *vg = static_cast<const T *>(a.v);
    float S[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!fresh) x = __ldcs(reinterpret_cast<const float4 *>(Sp + (g + 32 * i) * kDV));
        S[i][0] = x.x; S[i][1] = x.y; S[i][2] = x.z; S[i][3] = x.w;
    }
    // threads 0..127 fetch k (and alpha), 128..255 q, and 32 of them v
    float nx = 0.f, na = 0.f, nv = 0.f;
    auto fetch = [&](int t) {
        const int i = tid & (kDK - 1);
        if (tid < kDK) {
            nx = to_f(kg[t * a.stride_k + hq * kDK + i]);
            na = V == kKda ? a.alpha[((long long)t * a.heads + h) * kDK + i] : a.alpha[(long long)t * a.heads + h];
        } else {
            nx = to_f(qg[t * a.stride_q + hq * kDK + i]);
            if (i < kStepCols) nv = to_f(vg[t * a.stride_v + h * kDV + slice * kStepCols + i]);
        }
    };
    auto put = [&](int b) {
        const int i = tid & (kDK - 1);
        if (tid < kDK) {
            sk[b][i] = nx;
            sa[b][i] = na;
        } else {
            sq[b][i] = nx;
            if (i < kStepCols) sv[b][i] = nv;
        }
    };
    fetch(t0);
    put(0);
    __syncthreads();
    T *out = static_cast<T *>(a.out);
    int b = 0;
    for (int t = t0; t < t1; t++) {
        const int nb = b == 2 ? 0 : b + 1, e = t & 1;
        if (t + 1 < t1) fetch(t + 1);
        const float beta = a.beta[(long long)t * a.heads + h];
        float kk[4], p[4] = {}, o[4] = {}, kq = 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int row = g + 32 * i;
            kk[i] = sk[b][row];
            const float qq = sq[b][row], al = sa[b][row];
            kq = fmaf(kk[i], qq, kq);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                S[i][j] *= al;
                if (V != kLinear) p[j] = fmaf(S[i][j], kk[i], p[j]);
                o[j] = fmaf(S[i][j], qq, o[j]);
            }
        }
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) {
            kq += __shfl_xor_sync(kFull, kq, d);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (V != kLinear) p[j] += __shfl_xor_sync(kFull, p[j], d);
                o[j] += __shfl_xor_sync(kFull, o[j], d);
            }
        }
        if (l < 8) {
            *reinterpret_cast<float4 *>(&red[e][w][4 * c]) = make_float4(p[0], p[1], p[2], p[3]);
            *reinterpret_cast<float4 *>(&red[e][w][kStepCols + 4 * c]) = make_float4(o[0], o[1], o[2], o[3]);
            if (l == 0) red_kq[e][w] = kq;
        }
        if (t + 1 < t1) put(nb);
        __syncthreads();
        float u[4] = {sv[b][4 * c], sv[b][4 * c + 1], sv[b][4 * c + 2], sv[b][4 * c + 3]};
        if (V != kLinear) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float4 y = *reinterpret_cast<const float4 *>(&red[e][i][4 * c]);
                x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
            }
            u[0] -= x.x; u[1] -= x.y; u[2] -= x.z; u[3] -= x.w;
        }
#pragma unroll
        for (int j = 0; j < 4; j++) u[j] *= beta;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) S[i][j] = fmaf(kk[i], u[j], S[i][j]);
        if (tid < kStepCols) {
            // one thread a column: u of its own column, and the two sums over the warps
            float x = 0.f, y = 0.f, z = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                x += red[e][i][tid];
                y += red[e][i][kStepCols + tid];
                z += red_kq[e][i];
            }
            const float uu = beta * (V == kLinear ? sv[b][tid] : sv[b][tid] - x);
            out[((long long)t * a.heads + h) * kDV + slice * kStepCols + tid] = from_f<T>(fmaf(z, uu, y));
        }
        b = nb;
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
        __stcs(reinterpret_cast<float4 *>(Sp + (g + 32 * i) * kDV), make_float4(S[i][0], S[i][1], S[i][2], S[i][3]));
}

template <class T>
cudaError_t launch_steps_t(const PromptArgs &a, cudaStream_t s)
{
    const unsigned grid = (unsigned)a.p.requests * (unsigned)a.heads * kStepSlices;
    switch (a.variant) {
        case kGdn: k_prompt_steps<T, kGdn><<<grid, kStepThreads, 0, s>>>(a); break;
        case kKda: k_prompt_steps<T, kKda><<<grid, kStepThreads, 0, s>>>(a); break;
        default: k_prompt_steps<T, kLinear><<<grid, kStepThreads, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_steps(const PromptArgs &a, cudaStream_t s)
{
    if (a.p.requests == 0 || a.p.tokens == 0) return cudaSuccess;
    switch (a.dtype) {
        case kF32: return launch_steps_t<float>(a, s);
        case kF16: return launch_steps_t<__half>(a, s);
        default: return launch_steps_t<__nv_bfloat16>(a, s);
    }
}

}  // namespace stepq

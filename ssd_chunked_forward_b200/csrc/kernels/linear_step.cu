// linear_step.cu -- one token of linear attention for a batch of sequences:
// per (sequence b, head h), with l = exp(decay[h]),
//     h <- l h + k v^T,     y = scale q^T h.
//
// Bound by reading and writing the fp32 state once (8 K V bytes per chain; the
// vectors are 1/64 of that at K = V = 128), or by the launch when there are few
// chains.  A block takes up to 64 columns of one chain's state: a thread owns
// 4 of them (one when V is no multiple of 4) and the rows r0, r0 + nr, ...; it
// issues the loads of its rows before it touches the token's vectors, so that
// both latencies overlap.  q^T h of the rows a thread owns is added up over the
// row slices in shared memory, in a fixed order.
// Measured: 128 sequences, 80 heads, K = 128, V = 64: 105 us, 6.4 TB/s, 98 % of the
// copy rate; one sequence of 24 heads: 4 us of launch and latency.
#include "../common.cuh"
#include "../debug_checks.cuh"
#include "../linear.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;
constexpr int kRows = 8;  // rows in flight per thread

template <int VEC> struct Pack;
template <> struct Pack<4> { using type = float4; };
template <> struct Pack<1> { using type = float; };

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(const LinearStep p, int cols, int slices) {
    using P = typename Pack<VEC>::type;
    __shared__ float sK[256], sQ[256], sV[kCols];
    __shared__ float sY[kThreads * 4];
    const int bh = blockIdx.x / slices, sl = blockIdx.x % slices;
    const int b = bh / p.H, h = bh - b * p.H;
    const int c0 = sl * cols, cn = min(cols, p.V - c0);
    const int g = cols / VEC;          // threads across a row
    const int nr = kThreads / g;       // row slices
    const int tid = threadIdx.x;
    const int cc = (tid % g) * VEC, r0 = tid / g;
    const bool on = r0 < nr && cc < cn;
    float* hs = p.state + (long long)bh * p.K * p.V + c0 + cc;
    float hv[kRows][VEC];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int k = r0 + r * nr;
        if (on && k < p.K && SSD_INB(hs - p.state + (long long)k * p.V + VEC - 1, (long long)p.B * p.H * p.K * p.V))
            *reinterpret_cast<P*>(hv[r]) = *reinterpret_cast<const P*>(hs + (long long)k * p.V);
    }
    const T* q = (const T*)p.q.p + (long long)b * p.q.batch + (long long)(h / p.q.share) * p.q.head;
    const T* kp = (const T*)p.k.p + (long long)b * p.k.batch + (long long)(h / p.k.share) * p.k.head;
    const T* v = (const T*)p.v.p + (long long)b * p.v.batch + (long long)(h / p.v.share) * p.v.head;
    if (tid < p.K) {
        sK[tid] = to_f32(kp[tid]);
        sQ[tid] = to_f32(q[tid]);
    }
    if (tid < cn) sV[tid] = to_f32(v[c0 + tid]);
    const float2 lam = decay_power(p.decay[h], 1);
    __syncthreads();
    float acc[VEC] = {};
    if (on) {
        float vv[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) vv[c] = sV[cc + c];
        for (int kb = r0; kb < p.K; kb += kRows * nr) {
            if (kb > r0) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int k = kb + r * nr;
                    if (k < p.K && SSD_INB(hs - p.state + (long long)k * p.V + VEC - 1, (long long)p.B * p.H * p.K * p.V))
                        *reinterpret_cast<P*>(hv[r]) = *reinterpret_cast<const P*>(hs + (long long)k * p.V);
                }
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int k = kb + r * nr;
                if (k < p.K) {
                    const float kk = sK[k], qq = sQ[k];
#pragma unroll
                    for (int c = 0; c < VEC; ++c) {
                        hv[r][c] = fmaf(hv[r][c], lam.x, fmaf(hv[r][c], lam.y, kk * vv[c]));
                        acc[c] = fmaf(qq, hv[r][c], acc[c]);
                    }
                    if (SSD_INB(hs - p.state + (long long)k * p.V + VEC - 1, (long long)p.B * p.H * p.K * p.V))
                        *reinterpret_cast<P*>(hs + (long long)k * p.V) = *reinterpret_cast<const P*>(hv[r]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < VEC; ++c) sY[r0 * cols + cc + c] = acc[c];
    }
    __syncthreads();
    if (tid < cn) {
        float s = 0.f;
        for (int r = 0; r < nr; ++r) s += sY[r * cols + tid];
        const long long at = (long long)bh * p.V + c0 + tid;
        if (SSD_INB(at, (long long)p.B * p.H * p.V)) ((T*)p.y)[at] = from_f32<T>(p.scale * s);
    }
}

}  // namespace

cudaError_t launch_linear_step(const LinearStep& s, cudaStream_t st) {
    const bool vec = s.V % 4 == 0;
    const int slices = (s.V + kCols - 1) / kCols;
    const int per = (s.V + slices - 1) / slices;
    const int cols = vec ? (per + 3) / 4 * 4 : per;
    const long long grid = (long long)s.B * s.H * slices;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kernel = s.bf16 ? (vec ? linear_step_kernel<__nv_bfloat16, 4> : linear_step_kernel<__nv_bfloat16, 1>)
                         : (vec ? linear_step_kernel<float, 4> : linear_step_kernel<float, 1>);
    kernel<<<(unsigned)grid, kThreads, 0, st>>>(s, cols, slices);
    return cudaGetLastError();
}

}  // namespace ssd

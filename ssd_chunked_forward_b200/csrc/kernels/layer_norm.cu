// layer_norm.cu -- layer norm over each of the `groups` parts of a row (n =
// width / groups numbers), with an optional silu(gate) product behind it:
//     xh = (x - mean) rstd,  u = xh w + b,  y = u silu(z)
// and its backward,
//     du = dy silu(z),  dz = dy u silu'(z),  dxh = du w,
//     dx = rstd (dxh - mean(dxh) - xh mean(dxh xh)),
//     dw = sum over the rows of du xh,  db = sum over the rows of du.
//
// Bound by HBM: each tensor is read or written once.  A part of a row is held
// in the registers of a team of threads (a power of two of lanes when 32 are
// enough, else the whole block), so the variance is the mean of the squared
// distances from the mean, not a difference of sums.  A thread keeps its columns
// over all the rows of its block: weight and bias are loaded once, and the
// sums of dw and db stay in its registers; a block's sums are one row of
// `part`, and a second kernel adds those rows up in a fixed order, so the
// result does not depend on which block ran when.  The next row's loads are
// issued before the present row's reductions.
#include "../common.cuh"
#include "../debug_checks.cuh"
#include "../linear.h"

namespace ssd {
namespace {

template <int BYTES> struct RawBytes;
template <> struct RawBytes<16> { using type = uint4; };
template <> struct RawBytes<8> { using type = uint2; };
template <> struct RawBytes<4> { using type = uint32_t; };
template <> struct RawBytes<2> { using type = uint16_t; };

template <typename T, int VEC>
struct Vec {
    using Raw = typename RawBytes<VEC * sizeof(T)>::type;
    Raw raw;
    __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ void clear() { raw = Raw(); }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        T t[VEC];
        memcpy(t, &raw, sizeof(raw));
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = to_f32(t[i]);
    }
    static __device__ __forceinline__ void store(T* p, const float (&f)[VEC]) {
        T t[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) t[i] = from_f32<T>(f[i]);
        Raw r;
        memcpy(&r, t, sizeof(r));
        *reinterpret_cast<Raw*>(p) = r;
    }
};

// 1 / (1 + exp(-z)).  bf16 results take the special-function forms (relative
// error below 2^-20, against the result's 2^-9); fp32 results the exact ones.
template <typename T> __device__ __forceinline__ float sigmoid(float z);
template <> __device__ __forceinline__ float sigmoid<float>(float z) { return 1.f / (1.f + expf(-z)); }
template <> __device__ __forceinline__ float sigmoid<__nv_bfloat16>(float z) {
    return __fdividef(1.f, 1.f + ex2_approx(-1.4426950408889634f * z));
}

// the most threads that norm_shape() gives a block of this variant
constexpr int norm_threads(int vec, int nv) { return (vec == 4 && nv == 4) || nv == 16 ? 1024 : 512; }

// How the threads of a launch lie over rows and columns.
struct NormShape {
    int n;       // numbers in a part
    int team;    // threads of a part: a power of two up to 32, or the block
    int gpb;     // parts side by side in a block
    int slots;   // rows side by side in a block
    int slabs;   // blocks across a row
    int parts;   // blocks down the rows
    int threads;
};

// Sum of a and b over the team, in every thread of it.  Teams wider than a warp
// are the whole block; `turn` alternates the buffer so that one barrier per sum
// is enough.
__device__ __forceinline__ void team_sum(float& a, float& b, int team, int turn, float (*buf)[2][32]) {
    const int w = team < 32 ? team : 32;
    for (int o = w >> 1; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (team > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
        if (lane == 0) {
            buf[turn][0][warp] = a;
            buf[turn][1][warp] = b;
        }
        __syncthreads();
        a = lane < nw ? buf[turn][0][lane] : 0.f;
        b = lane < nw ? buf[turn][1][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    }
}

template <typename T, int VEC, int NV, bool GATE>
__global__ void __launch_bounds__(norm_threads(VEC, NV))
    layer_norm_kernel(const NormArgs a, const NormShape s) {
    __shared__ float buf[2][2][32];
    const int slab = blockIdx.x % s.slabs, part = blockIdx.x / s.slabs;
    const int tid = threadIdx.x, lane = tid % s.team, tm = tid / s.team;
    const int slot = tm / s.gpb, gl = tm - slot * s.gpb;
    const bool on = slot < s.slots;
    const int group = slab * s.gpb + gl;
    const float inv_n = 1.f / (float)s.n;
    float w[NV][VEC], b[NV][VEC];
    int col[NV];
    bool in[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (lane + v * s.team) * VEC;
        in[v] = on && c < s.n;
        col[v] = group * s.n + c;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            w[v][i] = a.weight && in[v] && SSD_INB(col[v] + i, a.width) ? a.weight[col[v] + i] : 1.f;
            b[v][i] = a.bias && in[v] && SSD_INB(col[v] + i, a.width) ? a.bias[col[v] + i] : 0.f;
        }
    }
    Vec<T, VEC> xr[NV], zr[NV];
    const long long step = (long long)s.parts * s.slots;
    auto fetch = [&](long long row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            xr[v].clear();
            if (GATE) zr[v].clear();
            if (in[v] && row < a.rows && SSD_INB(col[v] + VEC - 1, a.width)) {
                xr[v].load((const T*)a.x + row * a.x_stride + col[v]);
                if (GATE) zr[v].load((const T*)a.gate + row * a.gate_stride + col[v]);
            }
        }
    };
    int turn = 0;
    long long base = (long long)part * s.slots;
    fetch(base + slot);
    for (; base < a.rows; base += step) {
        const long long row = base + slot;
        float x[NV][VEC], z[NV][VEC];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            xr[v].get(x[v]);
            if (GATE) zr[v].get(z[v]);
        }
        fetch(row + step);
        float sum = 0.f, sq = 0.f, none = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum += x[v][i];
        team_sum(sum, none, s.team, turn, buf);
        turn ^= 1;
        const float mean = sum * inv_n;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[v][i] = in[v] ? x[v][i] - mean : 0.f;
                sq = fmaf(x[v][i], x[v][i], sq);
            }
        team_sum(sq, none, s.team, turn, buf);
        turn ^= 1;
        const float rstd = 1.f / sqrtf(fmaf(sq, inv_n, a.eps));
        if (row < a.rows && on) {
            if (a.stats && lane == 0) {
                const long long at = (row * a.groups + group) * 2;
                if (SSD_INB(at + 1, a.rows * a.groups * 2)) {
                    a.stats[at] = mean;
                    a.stats[at + 1] = rstd;
                }
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!in[v] || !SSD_INB(row * a.width + col[v] + VEC - 1, a.rows * a.width)) continue;
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    y[i] = fmaf(x[v][i] * rstd, w[v][i], b[v][i]);
                    if (GATE) y[i] *= z[v][i] * sigmoid<T>(z[v][i]);
                }
                Vec<T, VEC>::store((T*)a.y + row * a.width + col[v], y);
            }
        }
    }
}

template <typename T, int VEC, int NV, bool GATE>
__global__ void __launch_bounds__(norm_threads(VEC, NV))
    layer_norm_backward_kernel(const NormArgs a, const NormShape s) {
    extern __shared__ float sums[];  // [slots][cols of the block][2], when slots > 1
    __shared__ float buf[2][2][32];
    const int slab = blockIdx.x % s.slabs, part = blockIdx.x / s.slabs;
    const int tid = threadIdx.x, lane = tid % s.team, tm = tid / s.team;
    const int slot = tm / s.gpb, gl = tm - slot * s.gpb;
    const bool on = slot < s.slots;
    const int group = slab * s.gpb + gl;
    const float inv_n = 1.f / (float)s.n;
    float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
    int col[NV];
    bool in[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (lane + v * s.team) * VEC;
        in[v] = on && c < s.n;
        col[v] = group * s.n + c;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            w[v][i] = a.weight && in[v] && SSD_INB(col[v] + i, a.width) ? a.weight[col[v] + i] : 1.f;
            b[v][i] = GATE && a.bias && in[v] && SSD_INB(col[v] + i, a.width) ? a.bias[col[v] + i] : 0.f;
            dw[v][i] = db[v][i] = 0.f;
        }
    }
    Vec<T, VEC> xr[NV], dr[NV], zr[NV];
    float2 st = make_float2(0.f, 0.f);
    const long long step = (long long)s.parts * s.slots;
    auto fetch = [&](long long row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            xr[v].clear();
            dr[v].clear();
            if (GATE) zr[v].clear();
            if (in[v] && row < a.rows && SSD_INB(col[v] + VEC - 1, a.width)) {
                xr[v].load((const T*)a.x + row * a.x_stride + col[v]);
                dr[v].load((const T*)a.dy + row * a.dy_stride + col[v]);
                if (GATE) zr[v].load((const T*)a.gate + row * a.gate_stride + col[v]);
            }
        }
        const long long at = row * a.groups + group;
        if (on && row < a.rows && SSD_INB(at, a.rows * a.groups)) st = reinterpret_cast<const float2*>(a.stats)[at];
    };
    int turn = 0;
    long long base = (long long)part * s.slots;
    fetch(base + slot);
    for (; base < a.rows; base += step) {
        const long long row = base + slot;
        float xh[NV][VEC], dxh[NV][VEC];
        const float mean = st.x, rstd = st.y;
        const bool live = row < a.rows && on;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float x[VEC], d[VEC], z[VEC];
            xr[v].get(x);
            dr[v].get(d);
            if (GATE) zr[v].get(z);
            const bool use = in[v] && live;
            float dz[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float h = use ? (x[i] - mean) * rstd : 0.f;
                float du = d[i];
                if (GATE) {
                    const float sg = sigmoid<T>(z[i]);
                    dz[i] = d[i] * fmaf(h, w[v][i], b[v][i]) * (sg * fmaf(z[i], 1.f - sg, 1.f));
                    du *= z[i] * sg;
                }
                du = use ? du : 0.f;
                dw[v][i] = fmaf(du, h, dw[v][i]);
                db[v][i] += du;
                xh[v][i] = h;
                dxh[v][i] = du * w[v][i];
                s1 += dxh[v][i];
                s2 = fmaf(dxh[v][i], h, s2);
            }
            if (GATE && use && SSD_INB(row * a.width + col[v] + VEC - 1, a.rows * a.width))
                Vec<T, VEC>::store((T*)a.dgate + row * a.width + col[v], dz);
        }
        fetch(row + step);
        team_sum(s1, s2, s.team, turn, buf);
        turn ^= 1;
        s1 *= inv_n;
        s2 *= inv_n;
        if (live) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!in[v] || !SSD_INB(row * a.width + col[v] + VEC - 1, a.rows * a.width)) continue;
                float dx[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) dx[i] = rstd * (dxh[v][i] - s1 - xh[v][i] * s2);
                Vec<T, VEC>::store((T*)a.dx + row * a.width + col[v], dx);
            }
        }
    }
    if (!a.part) return;
    float* pw = a.part + (size_t)part * 2 * a.width;
    if (s.slots == 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (in[v] && SSD_INB(col[v] + i, a.width)) {
                    pw[col[v] + i] = dw[v][i];
                    pw[a.width + col[v] + i] = db[v][i];
                }
        return;
    }
    const int cols = s.gpb * s.n;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (in[v]) {
                const int c = col[v] + i - slab * cols;
                sums[(slot * 2) * cols + c] = dw[v][i];
                sums[(slot * 2 + 1) * cols + c] = db[v][i];
            }
    __syncthreads();
    for (int c = tid; c < 2 * cols; c += blockDim.x) {
        float t = 0.f;
        for (int k = 0; k < s.slots; ++k) t += sums[k * 2 * cols + c];
        const int cc = c < cols ? c : c - cols;
        if (SSD_INB(slab * cols + cc, a.width)) pw[(c < cols ? 0 : a.width) + slab * cols + cc] = t;
    }
}

// dweight and dbias: column c of part[p][0 or 1], added over p.  32 columns of
// one of the two by 8 slices of the rows per block.
__global__ void __launch_bounds__(256) norm_parts_kernel(const float* __restrict__ part, int parts, int width,
                                                         float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float s[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x, which = blockIdx.y;
    float t = 0.f;
    if (c < width)
        for (int p = y; p < parts; p += 8)
            if (SSD_INB(((long long)p * 2 + which) * width + c, (long long)parts * 2 * width))
                t += part[((size_t)p * 2 + which) * width + c];
    s[y][x] = t;
    __syncthreads();
    if (y == 0 && c < width) {
        for (int k = 1; k < 8; ++k) t += s[k][x];
        float* out = which ? dbias : dweight;
        if (out && SSD_INB(c, width)) out[c] = t;
    }
}

// Vector width, vectors per thread and the launch's shape.  A part of up to 32
// vectors is a team of lanes; wider ones take the block, with more vectors per
// thread only where 512 threads would not hold the part.
int norm_shape(long long rows, int width, int groups, bool bf16, int vec, NormShape* s, int* nv) {
    s->n = width / groups;
    const int v = (s->n + vec - 1) / vec;
    *nv = 1;
    if (v <= 32) {
        s->team = 1;
        while (s->team < v) s->team *= 2;
        const int teams = 256 / s->team;
        s->gpb = 1;
        for (int g = 1; g <= teams && g <= groups; ++g)
            if (groups % g == 0) s->gpb = g;
        s->slots = teams / s->gpb;
        if (s->slots > rows) s->slots = (int)rows;
        s->threads = (s->team * s->gpb * s->slots + 31) / 32 * 32;
    } else {
        const int most = vec == 1 ? 128 : 512;
        const int wide = vec == 1 ? 16 : 4;
        while (*nv < wide && (v + *nv - 1) / *nv > most) *nv *= vec == 1 ? 4 : 2;
        s->team = ((v + *nv - 1) / *nv + 31) / 32 * 32;
        s->gpb = s->slots = 1;
        s->threads = s->team;
    }
    s->slabs = groups / s->gpb;
    const int per_sm = 1024 / s->threads > 0 ? 1024 / s->threads : 1;
    long long parts = (148LL * per_sm + s->slabs - 1) / s->slabs;
    const long long most = (rows + s->slots - 1) / s->slots;
    s->parts = (int)(parts < most ? parts : most);
    return s->threads;
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p % bytes) == 0; }

// the widest vector that the part's length, the strides and the addresses allow
int norm_vec(const NormArgs& a) {
    const int e = a.bf16 ? 2 : 4;
    const int n = a.width / a.groups;
    for (int vec = 16 / e; vec >= 4; vec /= 2) {
        const int by = vec * e;
        if (n % vec || a.x_stride % vec || !aligned(a.x, by)) continue;
        if (a.gate && (a.gate_stride % vec || !aligned(a.gate, by))) continue;
        if (a.dy && (a.dy_stride % vec || !aligned(a.dy, by) || !aligned(a.dx, by))) continue;
        if (a.y && !aligned(a.y, by)) continue;
        if (a.dgate && !aligned(a.dgate, by)) continue;
        return vec;
    }
    return 1;
}

template <typename T, int VEC, int NV>
cudaError_t launch(const NormArgs& a, const NormShape& s, bool backward, cudaStream_t st) {
    const long long grid = (long long)s.slabs * s.parts;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (!backward) {
        if (a.gate) layer_norm_kernel<T, VEC, NV, true><<<(unsigned)grid, s.threads, 0, st>>>(a, s);
        else layer_norm_kernel<T, VEC, NV, false><<<(unsigned)grid, s.threads, 0, st>>>(a, s);
    } else {
        const size_t smem = s.slots > 1 ? (size_t)s.slots * 2 * s.gpb * s.n * sizeof(float) : 0;
        if (a.gate) layer_norm_backward_kernel<T, VEC, NV, true><<<(unsigned)grid, s.threads, smem, st>>>(a, s);
        else layer_norm_backward_kernel<T, VEC, NV, false><<<(unsigned)grid, s.threads, smem, st>>>(a, s);
    }
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_nv(const NormArgs& a, const NormShape& s, int nv, bool backward, cudaStream_t st) {
    if (nv == 1) return launch<T, VEC, 1>(a, s, backward, st);
    if constexpr (VEC == 1) {
        return nv == 4 ? launch<T, 1, 4>(a, s, backward, st) : launch<T, 1, 16>(a, s, backward, st);
    } else {
        return nv == 2 ? launch<T, VEC, 2>(a, s, backward, st) : launch<T, VEC, 4>(a, s, backward, st);
    }
}

cudaError_t launch_norm(const NormArgs& a, bool backward, cudaStream_t st) {
    NormShape s;
    int nv;
    const int vec = norm_vec(a);
    norm_shape(a.rows, a.width, a.groups, a.bf16, vec, &s, &nv);
    cudaError_t e;
    if (a.bf16)
        e = vec == 8 ? launch_nv<__nv_bfloat16, 8>(a, s, nv, backward, st)
          : vec == 4 ? launch_nv<__nv_bfloat16, 4>(a, s, nv, backward, st)
                     : launch_nv<__nv_bfloat16, 1>(a, s, nv, backward, st);
    else
        e = vec == 4 ? launch_nv<float, 4>(a, s, nv, backward, st) : launch_nv<float, 1>(a, s, nv, backward, st);
    if (e != cudaSuccess || !backward || !a.part) return e;
    const dim3 grid((a.width + 31) / 32, 2);
    norm_parts_kernel<<<grid, 256, 0, st>>>(a.part, s.parts, a.width, a.dweight, a.dbias);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t st) { return launch_norm(a, false, st); }

int norm_backward_parts(long long rows, int width, int groups, bool bf16) {
    int most = 1;
    for (int vec = bf16 ? 8 : 4; vec >= 1; vec = vec == 4 ? 1 : vec / 2) {
        NormShape s;
        int nv;
        norm_shape(rows, width, groups, bf16, vec, &s, &nv);
        if (s.parts > most) most = s.parts;
    }
    return most;
}

cudaError_t launch_layer_norm_backward(const NormArgs& a, cudaStream_t st) { return launch_norm(a, true, st); }

}  // namespace ssd

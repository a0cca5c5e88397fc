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
// result does not depend on which block ran when.
//
// The rows ahead are on their way into shared memory (cp.async, each thread the
// elements that it will read itself, so no barrier is needed) while a row is
// worked on, where one row in registers left the loads' latency in the open
// (32768 x 5120 in 80 groups, gate, forward: 227 us; with the ring 214).  What
// bounds the kernels beside HBM is issuing instructions: 72 % of the issue slots
// at 255 instructions for a vector of eight numbers, which is why arithmetic goes in
// pairs, pointers move along, and a thread takes more than one vector.
// Now: 32768 x 2560 forward 59.5 us (5.6 TB/s), backward 97 (5.2); 32768 x 5120 in 80
// groups with gate 164 (6.1) and 312 (5.4).  Elements of 2 bytes, which cp.async cannot copy, are
// prefetched one row ahead in registers.
#include <type_traits>

#include "../common.cuh"
#include "../debug_checks.cuh"
#include "../linear.h"
#include "../tc_common.cuh"

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

// Two fp32 numbers in one instruction: the kernels issue close to one instruction a
// cycle, and pairs halve the arithmetic's share (each number is rounded as ever).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}
// VEC numbers as pairs (one number: a pair whose second half is 0)
template <int VEC>
struct Pairs {
    static constexpr int N = (VEC + 1) / 2;
    float2 p[N];
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = make_float2(f[2 * i], 2 * i + 1 < VEC ? f[(2 * i + 1) % VEC] : 0.f);
    }
    __device__ __forceinline__ void out(float (&f)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = i & 1 ? p[i / 2].y : p[i / 2].x;
    }
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// rows ahead, by the vectors that a thread has of each: 196 KB at most
__host__ __device__ constexpr int norm_depth(int nv) { return nv == 1 ? 4 : nv == 2 ? 2 : 1; }

__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, std::integral_constant<int, 16>) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, std::integral_constant<int, 8>) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, std::integral_constant<int, 4>) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// A thread's elements of NT tensors in the rows ahead.  Slots are the thread's own.
template <typename T, int VEC, int NV, int NT>
struct Ahead {
    static constexpr int kBytes = VEC * (int)sizeof(T);
    static constexpr bool kRing = kBytes >= 4;
    static constexpr int kDepth = kRing ? norm_depth(NV) : 1;
    using V = Vec<T, VEC>;
    V held[kRing ? 1 : NT][kRing ? 1 : NV];
    uint8_t* mine;
    int pitch;
    // bytes of shared memory for a block of that many threads
    static size_t bytes(int threads) { return kRing ? (size_t)kDepth * NT * NV * threads * kBytes : 0; }
    __device__ __forceinline__ Ahead(uint8_t* smem) : mine(smem + threadIdx.x * kBytes), pitch(blockDim.x * kBytes) {}
    __device__ __forceinline__ uint8_t* slot(int stage, int t, int v) const {
        return mine + ((stage * NT + t) * NV + v) * pitch;
    }
    // src: the element's address, read only if `on`; else zeros come out
    __device__ __forceinline__ void issue(int stage, int t, int v, const T* src, bool on) {
        if constexpr (kRing) {
            if (on) {
                cp_async(static_cast<uint32_t>(__cvta_generic_to_shared(slot(stage, t, v))), src,
                         std::integral_constant<int, kBytes>());
            } else {
                V none;
                none.clear();
                *reinterpret_cast<typename V::Raw*>(slot(stage, t, v)) = none.raw;
            }
        } else {
            held[t][v].clear();
            if (on) held[t][v].load(src);
        }
    }
    __device__ __forceinline__ void commit() {
        if constexpr (kRing) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // the oldest row of kDepth is here
    __device__ __forceinline__ void wait() {
        if constexpr (kRing) asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    }
    __device__ __forceinline__ void get(int stage, int t, int v, Pairs<VEC>& to) const {
        float f[VEC];
        if constexpr (kRing) {
            V x;
            x.load(reinterpret_cast<const T*>(slot(stage, t, v)));
            x.get(f);
        } else {
            held[t][v].get(f);
        }
        to.set(f);
    }
};

// 1 / (1 + exp(-z)).  bf16 results take the special-function forms, against the result's
// own 2^-8: relative error at most (1.25 max(-z, 0) + 9) 2^-24 (the product in the exponent
// is rounded, and grows with -z; 2^-17 at -80), and 0 where 1 + exp(-z) passes 2^126
// (z < -87.3, silu above -2^-119); fp32 results take the exact ones.
template <typename T> __device__ __forceinline__ float sigmoid(float z);
template <> __device__ __forceinline__ float sigmoid<float>(float z) { return 1.f / (1.f + expf(-z)); }
template <> __device__ __forceinline__ float sigmoid<__nv_bfloat16>(float z) {
    return __fdividef(1.f, 1.f + ex2_approx(-1.4426950408889634f * z));
}

// the most threads that norm_shape() gives a block of this variant
constexpr int norm_threads(int vec, int nv) {
    return (vec == 4 && nv == 4) || nv == 16 ? 1024 : nv == 1 ? 256 : 512;
}

// How the threads of a launch lie over rows and columns.
struct NormShape {
    int n;       // numbers in a part
    int team;    // threads of a part: a power of two up to 32, or the block
    int gpb;     // parts side by side in a block
    int slots;   // rows side by side in a block
    int slabs;   // blocks across a row
    int parts;   // blocks down the rows
    int threads;
    int ring_bytes;  // of the rows ahead (the backward's moments lie behind them)
    long long most;  // blocks down the rows if each took one turn
    long long step;  // rows from one row of a thread to the next, and in numbers of each tensor
    long long x_step, gate_step, dy_step, out_step, stats_step;
};

// Sums of N numbers over the team, in every thread of it.  Teams wider than a warp
// are the whole block; the caller alternates between two buffers, so that one
// barrier per sum is enough.
template <int N>
__device__ __forceinline__ void team_sum(float (&a)[N], int team, float (*buf)[32]) {
    if (team >= 32) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
    } else {
        for (int o = team >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
    }
    if (team > 32) {
        const int nw = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) buf[i][threadIdx.x >> 5] = a[i];
        }
        __syncthreads();
        // four warps' sums to a read (those of no warp stay zero)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(&buf[i][0]), g = *reinterpret_cast<const float4*>(&buf[i][4]);
            a[i] = ((f.x + f.y) + (f.z + f.w)) + ((g.x + g.y) + (g.z + g.w));
        }
        for (int k = 8; k < nw; k += 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float4 f = *reinterpret_cast<const float4*>(&buf[i][k]);
                a[i] += (f.x + f.y) + (f.z + f.w);
            }
        }
    }
}

// x^(-1/2): the special-function unit's and one Newton step (within one rounding or
// two; the division and root that round exactly are forty instructions)
__device__ __forceinline__ float inv_sqrt(float x) {
    const float r = rsqrtf(x);
    return r > 0.f ? r * fmaf(-0.5f * x * r, r, 1.5f) : r;  // (squares that overflow: 0)
}

// The rows of a thread: row0, row0 + step, ..  Indices are counted in 32 bits and
// pointers moved along: with an index product for each access a row of 8 numbers
// cost a thread 255 instructions, now 140, and issuing them is what bounds
// these kernels next to HBM.
struct Rows {
    long long row0;
    int mine, all;  // rows of this thread, and of the block's first
    __device__ __forceinline__ Rows(const NormArgs& a, const NormShape& s, int part, int slot, bool on) {
        const long long first = (long long)part * s.slots;
        row0 = first + slot;
        all = first < a.rows ? (int)((a.rows - first + s.step - 1) / s.step) : 0;
        mine = on && row0 < a.rows ? (int)((a.rows - row0 + s.step - 1) / s.step) : 0;
    }
};

// A thread's place: its part of the row, its columns, and weight and bias there.
template <int VEC, int NV>
struct Place {
    int lane, slot, group, col[NV];
    bool on, in[NV];
    Pairs<VEC> w[NV], b[NV];
    __device__ __forceinline__ Place(const NormArgs& a, const NormShape& s, int slab, bool bias) {
        const int tid = threadIdx.x, tm = tid / s.team;
        lane = tid % s.team;
        slot = tm / s.gpb;
        on = slot < s.slots;
        group = slab * s.gpb + tm - slot * s.gpb;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + v * s.team) * VEC;
            in[v] = on && c < s.n;
            col[v] = group * s.n + c;
            float fw[VEC], fb[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                fw[i] = a.weight && in[v] && SSD_INB(col[v] + i, a.width) ? a.weight[col[v] + i] : 1.f;
                fb[i] = bias && a.bias && in[v] && SSD_INB(col[v] + i, a.width) ? a.bias[col[v] + i] : 0.f;
            }
            w[v].set(fw);
            b[v].set(fb);
        }
    }
};

template <typename T, int VEC, int NV, bool GATE>
__global__ void __launch_bounds__(norm_threads(VEC, NV), NV == 1 ? 4 : 1)
    layer_norm_kernel(const NormArgs a, const NormShape s) {
    __shared__ __align__(16) float buf[2][1][32];
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int P = Pairs<VEC>::N;
    using Ring = Ahead<T, VEC, NV, GATE ? 2 : 1>;
    constexpr int depth = Ring::kDepth;
    const int slab = blockIdx.x % s.slabs, part = blockIdx.x / s.slabs;
    const Place<VEC, NV> at(a, s, slab, true);
    for (int i = threadIdx.x; i < 64; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
    __syncthreads();
    const float inv_n = 1.f / (float)s.n;
    const Rows rows(a, s, part, at.slot, at.on);
    Ring ring(smem);
    const int next = s.team * VEC;  // from one vector of a thread to the next
    const T* px = (const T*)a.x + rows.row0 * a.x_stride + at.col[0];
    const T* pz = (const T*)a.gate + rows.row0 * a.gate_stride + at.col[0];
    T* py = (T*)a.y + rows.row0 * a.width + at.col[0];
    float2* pst = a.stats ? reinterpret_cast<float2*>(a.stats) + rows.row0 * a.groups + at.group : nullptr;
    auto fetch = [&](int k, int stage) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool use = at.in[v] && k < rows.mine &&
                             SSD_INB((rows.row0 + k * s.step) * a.width + at.col[v] + VEC - 1, a.rows * a.width);
            ring.issue(stage, 0, v, px + v * next, use);
            if (GATE) ring.issue(stage, 1, v, pz + v * next, use);
        }
        px += s.x_step;
        if (GATE) pz += s.gate_step;
        ring.commit();
    };
    int stage = 0;
#pragma unroll
    for (int i = 0; i < depth; ++i) fetch(i, i);
    for (int k = 0; k < rows.all; ++k) {
        Pairs<VEC> x[NV], z[NV];
        ring.wait();
        float2 t = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            ring.get(stage, 0, v, x[v]);
            if (GATE) ring.get(stage, 1, v, z[v]);
#pragma unroll
            for (int i = 0; i < P; ++i) t = add2(t, x[v].p[i]);  // (zeros behind the part)
        }
        fetch(k + depth, stage);
        stage = stage + 1 == depth ? 0 : stage + 1;
        float sum[1] = {t.x + t.y};
        team_sum(sum, s.team, buf[0]);
        const float mean = sum[0] * inv_n;
        t = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const float2 away = both(at.in[v] ? -mean : 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                x[v].p[i] = add2(x[v].p[i], away);
                if (VEC == 1) x[v].p[i].y = 0.f;
                t = tc::fma2(x[v].p[i], x[v].p[i], t);
            }
        }
        float sq[1] = {t.x + t.y};
        team_sum(sq, s.team, buf[1]);
        const float rstd = inv_sqrt(fmaf(sq[0], inv_n, a.eps));
        if (k < rows.mine) {
            if (pst && at.lane == 0 && SSD_INB((float*)pst - a.stats + 1, a.rows * a.groups * 2)) *pst = make_float2(mean, rstd);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!at.in[v] || !SSD_INB(py + v * next - (T*)a.y + VEC - 1, a.rows * a.width)) continue;
                Pairs<VEC> y;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    y.p[i] = tc::fma2(tc::mul2(x[v].p[i], both(rstd)), at.w[v].p[i], at.b[v].p[i]);
                    if (GATE) {
                        const float2 sg = make_float2(sigmoid<T>(z[v].p[i].x), sigmoid<T>(z[v].p[i].y));
                        y.p[i] = tc::mul2(y.p[i], tc::mul2(z[v].p[i], sg));
                    }
                }
                float f[VEC];
                y.out(f);
                Vec<T, VEC>::store(py + v * next, f);
            }
        }
        py += s.out_step;
        if (pst) pst += s.stats_step;
    }
}

template <typename T, int VEC, int NV, bool GATE>
__global__ void __launch_bounds__(norm_threads(VEC, NV), NV == 1 ? 2 : 1)
    layer_norm_backward_kernel(const NormArgs a, const NormShape s) {
    extern __shared__ __align__(16) uint8_t smem[];
    next_may_start();
    float* sums = reinterpret_cast<float*>(smem);  // at the end: [slots][2][cols of the block], when slots > 1
    __shared__ __align__(16) float buf[2][2][32];
    constexpr int P = Pairs<VEC>::N, NT = GATE ? 3 : 2;
    using Ring = Ahead<T, VEC, NV, NT>;
    constexpr int depth = Ring::kDepth;
    const int slab = blockIdx.x % s.slabs, part = blockIdx.x / s.slabs;
    const Place<VEC, NV> at(a, s, slab, GATE);
    for (int i = threadIdx.x; i < 128; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
    __syncthreads();
    const float inv_n = 1.f / (float)s.n;
    Pairs<VEC> dw[NV], db[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < P; ++i) dw[v].p[i] = db[v].p[i] = both(0.f);
    const Rows rows(a, s, part, at.slot, at.on);
    Ring ring(smem);
    // mean and rstd of the part go with the rows ahead
    float2* moments = reinterpret_cast<float2*>(smem + s.ring_bytes) + threadIdx.x;
    float2 held = make_float2(0.f, 0.f);
    const int next = s.team * VEC;
    const T* px = (const T*)a.x + rows.row0 * a.x_stride + at.col[0];
    const T* pd = (const T*)a.dy + rows.row0 * a.dy_stride + at.col[0];
    const T* pz = (const T*)a.gate + rows.row0 * a.gate_stride + at.col[0];
    const float2* pst = reinterpret_cast<const float2*>(a.stats) + rows.row0 * a.groups + at.group;
    long long to = rows.row0 * a.width + at.col[0];  // in dx and dgate
    auto fetch = [&](int k, int stage) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool use = at.in[v] && k < rows.mine &&
                             SSD_INB((rows.row0 + k * s.step) * a.width + at.col[v] + VEC - 1, a.rows * a.width);
            ring.issue(stage, 0, v, px + v * next, use);
            ring.issue(stage, 1, v, pd + v * next, use);
            if (GATE) ring.issue(stage, 2, v, pz + v * next, use);
        }
        const bool use = k < rows.mine && SSD_INB((const float*)pst - a.stats + 1, a.rows * a.groups * 2);
        if constexpr (Ring::kRing) {
            if (use)
                cp_async(static_cast<uint32_t>(__cvta_generic_to_shared(moments + stage * blockDim.x)), pst,
                         std::integral_constant<int, 8>());
            else
                moments[stage * blockDim.x] = make_float2(0.f, 0.f);
        } else {
            held = use ? *pst : make_float2(0.f, 0.f);
        }
        px += s.x_step;
        pd += s.dy_step;
        if (GATE) pz += s.gate_step;
        pst += s.stats_step;
        ring.commit();
    };
    int turn = 0, stage = 0;
#pragma unroll
    for (int i = 0; i < depth; ++i) fetch(i, i);
    for (int k = 0; k < rows.all; ++k) {
        const bool live = k < rows.mine;
        Pairs<VEC> xh[NV], dxh[NV];
        ring.wait();
        if constexpr (Ring::kRing) held = moments[stage * blockDim.x];
        const float rstd = held.y;
        float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            Pairs<VEC> x, d, z, dz;
            ring.get(stage, 0, v, x);
            ring.get(stage, 1, v, d);
            if (GATE) ring.get(stage, 2, v, z);
            const float2 away = both(at.in[v] ? -held.x : 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                // zeros behind the part and the last row: dy = 0 there, so they add nothing
                const float2 h = tc::mul2(add2(x.p[i], away), both(rstd));
                float2 du = d.p[i];
                if (GATE) {
                    const float2 sg = make_float2(sigmoid<T>(z.p[i].x), sigmoid<T>(z.p[i].y));
                    const float2 zs = tc::mul2(z.p[i], sg);  // silu(z); silu'(z) = sg + zs (1 - sg)
                    const float2 slope = tc::fma2(zs, add2(both(1.f), make_float2(-sg.x, -sg.y)), sg);
                    dz.p[i] = tc::mul2(tc::mul2(du, slope), tc::fma2(h, at.w[v].p[i], at.b[v].p[i]));
                    du = tc::mul2(du, zs);
                }
                dw[v].p[i] = tc::fma2(du, h, dw[v].p[i]);
                db[v].p[i] = add2(db[v].p[i], du);
                xh[v].p[i] = h;
                dxh[v].p[i] = tc::mul2(du, at.w[v].p[i]);
                s1 = add2(s1, dxh[v].p[i]);
                s2 = tc::fma2(dxh[v].p[i], h, s2);
            }
            if (GATE && at.in[v] && live && SSD_INB(to + v * next + VEC - 1, a.rows * a.width)) {
                float f[VEC];
                dz.out(f);
                Vec<T, VEC>::store((T*)a.dgate + to + v * next, f);
            }
        }
        fetch(k + depth, stage);
        stage = stage + 1 == depth ? 0 : stage + 1;
        float both_sums[2] = {s1.x + s1.y, s2.x + s2.y};
        team_sum(both_sums, s.team, buf[turn]);
        turn ^= 1;
        if (live) {
            const float2 m1 = both(-both_sums[0] * inv_n), m2 = both(-both_sums[1] * inv_n);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!at.in[v] || !SSD_INB(to + v * next + VEC - 1, a.rows * a.width)) continue;
                Pairs<VEC> dx;
#pragma unroll
                for (int i = 0; i < P; ++i)
                    dx.p[i] = tc::mul2(both(rstd), tc::fma2(xh[v].p[i], m2, add2(dxh[v].p[i], m1)));
                float f[VEC];
                dx.out(f);
                Vec<T, VEC>::store((T*)a.dx + to + v * next, f);
            }
        }
        to += s.out_step;
    }
    if (!a.part) return;
    float* pw = a.part + (size_t)part * 2 * a.width;
    const int cols = s.gpb * s.n;
    if (s.slots > 1) __syncthreads();  // every slot of the ring has been read
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float fw[VEC], fb[VEC];
        dw[v].out(fw);
        db[v].out(fb);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if (!at.in[v] || !SSD_INB(at.col[v] + i, a.width)) continue;
            if (s.slots == 1) {
                pw[at.col[v] + i] = fw[i];
                pw[a.width + at.col[v] + i] = fb[i];
            } else {
                const int c = at.col[v] + i - slab * cols;
                sums[(at.slot * 2) * cols + c] = fw[i];
                sums[(at.slot * 2 + 1) * cols + c] = fb[i];
            }
        }
    }
    if (s.slots == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * cols; c += blockDim.x) {
        float t = 0.f;
        for (int k = 0; k < s.slots; ++k) t += sums[k * 2 * cols + c];
        const int cc = c < cols ? c : c - cols;
        if (SSD_INB(slab * cols + cc, a.width)) pw[(c < cols ? 0 : a.width) + slab * cols + cc] = t;
    }
}

// dweight and dbias: column c of part[p][0 or 1], added over p.  32 columns of
// one of the two by 8 slices of the rows per block.
__global__ void __launch_bounds__(256) norm_parts_kernel(const float* part, int parts, int width, float* dweight,
                                                         float* dbias) {
    __shared__ float s[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = (blockIdx.x >> 1) * 32 + x, which = blockIdx.x & 1;
    wait_for_earlier();
    float t = 0.f;
    if (c < width)
        for (int p = y; p < parts; p += 8)
            if (SSD_INB(((long long)p * 2 + which) * width + c, (long long)parts * 2 * width))
                t += __ldcg(part + ((size_t)p * 2 + which) * width + c);
    s[y][x] = t;
    __syncthreads();
    if (y == 0 && c < width) {
        for (int k = 1; k < 8; ++k) t += s[k][x];
        float* out = which ? dbias : dweight;
        if (out && SSD_INB(c, width)) out[c] = t;
    }
}

// Blocks down the rows where an SM holds `resident` of them: one more than fit would
// keep the others waiting for a second turn (32768 x 5120 in 80 groups: 166 us with
// 296 blocks, 242 with 300).
int norm_parts(const NormShape& s, int resident) {
    const long long parts = 148LL * (resident > 0 ? resident : 1) / s.slabs;
    return (int)(parts < 1 ? 1 : parts < s.most ? parts : s.most);
}

// Vectors per thread and the launch's shape.  What a row costs a thread beside its
// numbers (sums, barriers, counting) is shared by all of them, so a thread takes two
// vectors of a part (32768 x 2560: forward 71 us, with one 89; backward 104, with one
// 137; 20000 x 2560 in 32 groups: 54 and 69, backward 78 and 102).  Exceptions:
//   the gated backward of narrow parts in vectors of eight, whose three tensors then
//     spill registers.  Two against one vector, time: 1.27 at 16384 x 2048 in 64 groups,
//     1.10 at 16384 x 1536 in 24 (58.4 us with one), 1.12 at 4096 x 5120 in 80, 1.09 at
//     32768 x 2048 in 16; even at 65536 x 640 in 8; 0.97 to 0.99 from 80 million numbers on
//     (32768 x 5120 in 80: 302 and 312 us).  Vectors of four do not spill: bf16
//     0.76 at 65536 x 800 in 8 and 0.70 at 20000 x 1440 in 40, fp32 0.80 at 65536 x 640 in
//     8, 0.96 at 32768 x 2560 in 80, 1.03 at most (8192 x 1536 in 24);
//   the plain forward of bf16 parts of more than 384 vectors takes four.  Four against
//     two: 0.76 at 16384 x 8192 (98 us), 0.78 at x 6144, 0.97 at x 5120, 0.94 at x 3200, 0.91
//     at 32768 x 4096; 1.06 at 4096 x 4096.  (Gated 229 us with four, 178 with two);
//   what the block could not hold otherwise.
// A part of up to 32 threads is a team of lanes, and a block takes the parts and rows
// that leave an SM's threads busiest; wider parts take a block each.
void norm_shape(long long rows, int width, int groups, int vec, bool gate, bool backward, NormShape* s, int* nv) {
    s->n = width / groups;
    const int v = (s->n + vec - 1) / vec;
    *nv = vec > 2 && v >= 4 && (v > 32 || vec < 8 || !(backward && gate)) ? 2 : 1;
    // threads that an SM holds at the kernels' registers
    const int hold = *nv == 1 && !backward ? 1024 : 512;
    if ((v + *nv - 1) / *nv <= 32) {
        s->team = 1;
        while (s->team * *nv < v) s->team *= 2;
        int best = 0;
        for (int g = 1; g * s->team <= 256 && g <= groups; ++g) {
            if (groups % g) continue;
            for (int k = 1; k * g * s->team <= 256 && k <= rows; ++k) {
                const int threads = (k * g * s->team + 31) / 32 * 32;
                const int busy = hold / threads * (k * g * s->team);
                if (busy < best) continue;
                best = busy;
                s->gpb = g;
                s->slots = k;
                s->threads = threads;
            }
        }
    } else {
        const int wide = vec <= 2 ? 16 : 4;
        auto most = [&] {  // threads of a block before each takes more vectors
            if (vec <= 2) return *nv == 1 ? 128 : 512;
            return backward || gate || vec < 8 ? 512 : 192;
        };
        while (*nv < wide && (v + *nv - 1) / *nv > most()) *nv *= vec <= 2 ? 4 : 2;
        s->team = ((v + *nv - 1) / *nv + 31) / 32 * 32;
        s->gpb = s->slots = 1;
        s->threads = s->team;
    }
    s->slabs = groups / s->gpb;
    s->most = (rows + s->slots - 1) / s->slots;
    s->parts = norm_parts(*s, (backward ? 1024 : 512) / s->threads);
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p % bytes) == 0; }

// the widest vector that the part's length, the strides and the addresses allow
int norm_vec(const NormArgs& a) {
    const int e = a.bf16 ? 2 : 4;
    const int n = a.width / a.groups;
    for (int vec = 16 / e; vec >= 2; vec /= 2) {
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
cudaError_t launch(const NormArgs& a, NormShape& s, bool backward, cudaStream_t st) {
    const int tensors = (a.gate ? 2 : 1) + (backward ? 1 : 0);
    size_t smem = tensors == 1   ? Ahead<T, VEC, NV, 1>::bytes(s.threads)
                  : tensors == 2 ? Ahead<T, VEC, NV, 2>::bytes(s.threads)
                                 : Ahead<T, VEC, NV, 3>::bytes(s.threads);
    s.ring_bytes = (int)smem;
    if (backward) {
        smem += (size_t)norm_depth(NV) * s.threads * sizeof(float2);
        const size_t sums = s.slots > 1 ? (size_t)s.slots * 2 * s.gpb * s.n * sizeof(float) : 0;
        if (smem < sums) smem = sums;
    }
    auto kernel = backward ? (a.gate ? layer_norm_backward_kernel<T, VEC, NV, true> : layer_norm_backward_kernel<T, VEC, NV, false>)
                           : (a.gate ? layer_norm_kernel<T, VEC, NV, true> : layer_norm_kernel<T, VEC, NV, false>);
    if (smem > 40 * 1024) {  // (some KB are static)
        cudaError_t e = allow_smem(kernel, 1024);
        if (e != cudaSuccess) return e;
    }
    if (s.most * s.slabs > 148) {
        int resident = 1;
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, s.threads, smem);
        if (e != cudaSuccess) return e;
        int parts = norm_parts(s, resident);
        // The gated bf16 forward over narrow parts starts new blocks after 64 rows of a thread.
        // Time against blocks that stay: 0.92 at 65536 x 5120 in 80 groups (352 us if they
        // stay), 0.95 at 32768 x and 0.97 at 24576 x, 0.97 at 131072 x 1536 in 24, 0.98 at 16384
        // x 5120, 1.03 at 20000 x 1440 in 40.  The others keep theirs: 1.02 to 1.04 without a gate and for wide parts (65536
        // x 2560, 131072 x 2560, 65536 x 2048 in 16, 32768 x 4096 gated), 0.97 to 1.03 in fp32.
        if (!backward && a.gate && a.bf16 && s.team <= 32)
            parts = norm_parts(s, resident * (1 + (int)(s.most / parts / 64)));
        s.parts = backward && parts > s.parts ? s.parts : parts;  // (the workspace holds that many)
    }
    s.step = (long long)s.parts * s.slots;
    s.x_step = s.step * a.x_stride;
    s.gate_step = s.step * a.gate_stride;
    s.dy_step = s.step * a.dy_stride;
    s.out_step = s.step * a.width;
    s.stats_step = s.step * a.groups;
    const long long grid = (long long)s.slabs * s.parts;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    kernel<<<(unsigned)grid, s.threads, smem, st>>>(a, s);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_nv(const NormArgs& a, NormShape& s, int nv, bool backward, cudaStream_t st) {
    if (nv == 1) return launch<T, VEC, 1>(a, s, backward, st);
    if constexpr (VEC <= 2) {
        return nv == 4 ? launch<T, VEC, 4>(a, s, backward, st) : launch<T, VEC, 16>(a, s, backward, st);
    } else {
        return nv == 2 ? launch<T, VEC, 2>(a, s, backward, st) : launch<T, VEC, 4>(a, s, backward, st);
    }
}

cudaError_t launch_norm(const NormArgs& a, bool backward, cudaStream_t st) {
    NormShape s;
    int nv;
    const int vec = norm_vec(a);
    norm_shape(a.rows, a.width, a.groups, vec, a.gate, backward, &s, &nv);
    cudaError_t e;
    if (a.bf16)
        e = vec == 8 ? launch_nv<__nv_bfloat16, 8>(a, s, nv, backward, st)
          : vec == 4 ? launch_nv<__nv_bfloat16, 4>(a, s, nv, backward, st)
          : vec == 2 ? launch_nv<__nv_bfloat16, 2>(a, s, nv, backward, st)
                     : launch_nv<__nv_bfloat16, 1>(a, s, nv, backward, st);
    else
        e = vec == 4   ? launch_nv<float, 4>(a, s, nv, backward, st)
            : vec == 2 ? launch_nv<float, 2>(a, s, nv, backward, st)
                       : launch_nv<float, 1>(a, s, nv, backward, st);
    if (e != cudaSuccess || !backward || !a.part) return e;
    return launch_in_call(norm_parts_kernel, (unsigned)((a.width + 31) / 32 * 2), 256, 0, st, true,
                          (const float*)a.part, s.parts, a.width, a.dweight, a.dbias);
}

}  // namespace

cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t st) { return launch_norm(a, false, st); }

int norm_backward_parts(long long rows, int width, int groups, bool bf16) {
    int most = 1;
    for (int vec = bf16 ? 8 : 4; vec >= 1; vec /= 2) {
        for (int gate = 0; gate < 2; ++gate) {
            NormShape s;
            int nv;
            norm_shape(rows, width, groups, vec, gate, true, &s, &nv);
            if (s.parts > most) most = s.parts;
        }
    }
    return most;
}

cudaError_t launch_layer_norm_backward(const NormArgs& a, cudaStream_t st) { return launch_norm(a, true, st); }

}  // namespace ssd

// linear_simt.cu -- the linear-attention scan on CUDA cores (fp32 arithmetic,
// any sizes up to 256, any strides), the combination of the states of cut
// chains, and the sum of a shared head's gradients over its query heads.
//
// One block per (item, 64 columns of the state).  Chunks of 32 tokens: with
// positions i, j in the chunk, n tokens in it, H the state entering it and
// l = exp(decay),
//     out_i = sum_{j<=i} l^(i-j) (q_i.k_j) v_j + l^(i+1) q_i^T H
//     H    <- l^n H + sum_j l^(n-1-j) k_j v_j^T
// and the mirror image of it for a scan backwards.  The chunk's rows and H are
// in shared memory as fp32; every product is a small register tile.  32 tokens
// keep the masked quadratic part small next to the two state products, which
// are the operator's own work (2 K V multiply-adds per token and head).
//
// Bound by the fp32 pipes and the shared-memory reads that feed them; short calls
// by the latency of a chunk (some 4 us). Measured, fp32: 4 x 2048 tokens, 16 heads,
// 64 x 128 567 us (gradients 1460); 2 x 333 tokens, 8 query and 2 key heads, 48 x 64
// 33 (gradients 54); bf16, 8 x 700 tokens, 24 heads, 100 x 100 607 (gradients 1504).
#include "../common.cuh"
#include "../debug_checks.cuh"
#include "../linear.h"

namespace ssd {
namespace {

constexpr int kC = kSimtChunk;     // tokens of a chunk
constexpr int kVT = kSimtColumns;  // state columns of a block
constexpr int kThreads = 256;

// rows [t, t+n) of a tensor, D of its columns from c0 on, into fp32 rows of
// pitch ld; the rows behind n and the columns behind D up to Dp are zero
template <typename T>
__device__ void load_rows(const RowTensor& a, const ScanItem& it, int t, int n, int c0, int D, int Dp, int ld,
                          float* dst, long long rows, long long batches) {
    const T* base = (const T*)a.p + (long long)it.batch * a.batch + (long long)(it.head / a.share) * a.head + c0;
    // four loads on their way together, of four numbers where the rows allow it
    constexpr int U = 4;
    const bool four = ((D | Dp) & 3) == 0 && ((a.token | a.head | a.batch | c0) & 3) == 0 &&
                      (uintptr_t)a.p % (4 * sizeof(T)) == 0;
    if (four) {
        const int per = Dp / 4;
        for (int e0 = threadIdx.x; e0 < kC * per; e0 += U * kThreads) {
            float4 v[U];
            int at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + u * kThreads, r = e / per, c = 4 * (e - r * per);
                const long long row = it.row0 + t + r;
                at[u] = r * ld + c;
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < n && c < D && SSD_INB(row, rows) && SSD_INB(it.batch, batches)) {
                    const T* p = base + row * a.token + c;
                    if constexpr (sizeof(T) == 4) {
                        v[u] = *reinterpret_cast<const float4*>(p);
                    } else {
                        const uint2 b = *reinterpret_cast<const uint2*>(p);
                        v[u] = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                                           __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e0 + u * kThreads < kC * per) *reinterpret_cast<float4*>(dst + at[u]) = v[u];
        }
        return;
    }
    for (int e0 = threadIdx.x; e0 < kC * Dp; e0 += U * kThreads) {
        float v[U];
        int at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * kThreads, r = e / Dp, c = e - r * Dp;
            const long long row = it.row0 + t + r;
            at[u] = r * ld + c;
            v[u] = 0.f;
            if (r < n && c < D && SSD_INB(row, rows) && SSD_INB(it.batch, batches)) v[u] = to_f32(base[row * a.token + c]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (e0 + u * kThreads < kC * Dp) dst[at[u]] = v[u];
    }
}

template <typename T, bool kOut>
__global__ void __launch_bounds__(kThreads) scan_simt_kernel(const ScanLaunch p, int ntiles) {
    extern __shared__ __align__(16) float sm[];
    __shared__ ScanItem sItem;
    next_may_start();
    if (p.reset && blockIdx.x == 0 && threadIdx.x == 0) *p.status = kDevOk;
    if (threadIdx.x < 32) {
        ScanItem it = scan_item(p.plan, blockIdx.x / ntiles);
        if (it.valid) scan_item_tokens(it, p.plan.seg_tokens, p.role[it.role].reverse);
        if (threadIdx.x == 0) sItem = it;
    }
    __syncthreads();
    wait_for_earlier();
    const ScanItem it = sItem;
    if (!it.valid || (!kOut && it.seg == it.nseg - 1)) return;
    const ScanRole& R = p.role[it.role];
    const int K = R.K, V = R.V, H = p.plan.H;
    const int v0 = (blockIdx.x % ntiles) * kVT;
    if (v0 >= V) return;
    const int vn = min(kVT, V - v0);
    const SimtLayout L = simt_layout(K);
    float* sQ = sm;
    float* sK = sQ + kC * L.ldk;
    float* sV = sK + kC * L.ldk;            // [kC][kVT]
    float* sP = sV + kC * kVT;              // [kC][kC + 4]
    float* sH = sP + kC * (kC + 4);         // [K4][kVT]
    float* sTab = sH + L.K4 * kVT;          // l^0 .. l^kC
    const int tid = threadIdx.x;
    const float la = p.decay[it.head];
    for (int d = tid; d <= kC; d += kThreads) sTab[d] = decay_power(la, d).x;
    const long long rows = p.plan.T, batches = p.plan.packed ? 1 : p.plan.B;
    (void)batches;
    const long long chain = (long long)it.seq * H + it.head;
    const long long chains = (long long)p.plan.B * H;

    // the state entering the item
    const bool from_init = it.slot_prev < 0;
    for (int e = tid; e < L.K4 * kVT; e += kThreads) {
        const int k = e / kVT, c = e % kVT;
        float h = 0.f;
        if (kOut && k < K && c < vn) {
            if (!from_init && (it.seg > 0 || R.init)) {
                const long long at = it.slot_prev * K * V + (long long)k * V + v0 + c;
                if (SSD_INB(at, p.plan.slots() * K * V)) h = p.states[at];
            } else if (from_init && R.init) {
                const long long at = chain * K * V + k * R.init_k + (v0 + c) * R.init_v;
                if (SSD_INB(at, chains * K * V)) h = R.init[at] * R.init_scale;
            }
        }
        sH[e] = h;
    }
    // a backward scan's initial state meets its first token undecayed
    int off = (it.seg == 0 && R.reverse) ? 0 : 1;
    const int span = it.t1 - it.t0, nch = (span + kC - 1) / kC;
    const float2 full = decay_power(la, kC);
    const int cg = (tid & 15) * 4;  // 4 columns
    const int rg = tid >> 4;        // 16 row groups

    for (int c = 0; c < nch; ++c) {
        const int ct = it.t0 + (R.reverse ? nch - 1 - c : c) * kC;
        const int n = min(kC, it.t1 - ct);
        __syncthreads();
        if (kOut) load_rows<T>(R.q, it, ct, n, 0, K, L.K4, L.ldk, sQ, rows, batches);
        load_rows<T>(R.k, it, ct, n, 0, K, L.K4, L.ldk, sK, rows, batches);
        load_rows<T>(R.v, it, ct, n, v0, vn, kVT, kVT, sV, rows, batches);
        __syncthreads();
        if (kOut) {
            // scores: row i, columns j0 + 8 m
            const int i = tid >> 3, j0 = tid & 7;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < L.K4; k += 4) {
                const float4 a = *reinterpret_cast<const float4*>(sQ + i * L.ldk + k);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float4 b = *reinterpret_cast<const float4*>(sK + (j0 + 8 * m) * L.ldk + k);
                    s[m] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s[m]))));
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int j = j0 + 8 * m, d = R.reverse ? j - i : i - j;
                sP[i * (kC + 4) + j] = (d >= 0 && i < n && j < n) ? s[m] * sTab[d] : 0.f;
            }
            __syncthreads();
            // rows 2 rg, 2 rg + 1; columns cg .. cg + 3
            float inter[2][4] = {}, intra[2][4] = {};
            const int i0 = 2 * rg;
            for (int k = 0; k < L.K4; k += 4) {
                float qa[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    *reinterpret_cast<float4*>(qa[r]) = *reinterpret_cast<const float4*>(sQ + (i0 + r) * L.ldk + k);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const float4 h = *reinterpret_cast<const float4*>(sH + (k + kk) * kVT + cg);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        inter[r][0] = fmaf(qa[r][kk], h.x, inter[r][0]);
                        inter[r][1] = fmaf(qa[r][kk], h.y, inter[r][1]);
                        inter[r][2] = fmaf(qa[r][kk], h.z, inter[r][2]);
                        inter[r][3] = fmaf(qa[r][kk], h.w, inter[r][3]);
                    }
                }
            }
            for (int j = 0; j < kC; j += 4) {
                float pa[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    *reinterpret_cast<float4*>(pa[r]) =
                        *reinterpret_cast<const float4*>(sP + (i0 + r) * (kC + 4) + j);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const float4 v = *reinterpret_cast<const float4*>(sV + (j + kk) * kVT + cg);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        intra[r][0] = fmaf(pa[r][kk], v.x, intra[r][0]);
                        intra[r][1] = fmaf(pa[r][kk], v.y, intra[r][1]);
                        intra[r][2] = fmaf(pa[r][kk], v.z, intra[r][2]);
                        intra[r][3] = fmaf(pa[r][kk], v.w, intra[r][3]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i1 = i0 + r;
                if (i1 >= n) continue;
                // a masked score is a zero, but 0 v of an infinity or NaN is one: then only
                // the causal side again
                float zero = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) zero = fmaf(intra[r][q], 0.f, zero);
                if (!(zero == 0.f)) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) intra[r][q] = 0.f;
                    for (int j = R.reverse ? i1 : 0; j < (R.reverse ? n : i1 + 1); ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            intra[r][q] = fmaf(sP[i1 * (kC + 4) + j], sV[j * kVT + cg + q], intra[r][q]);
                }
                const float e = sTab[(R.reverse ? n - 1 - i1 : i1) + off];
                const long long row = (long long)it.batch * rows + it.row0 + ct + i1;
                const long long at = (row * H + it.head) * V + v0 + cg;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (cg + q >= vn || !SSD_INB(at + q, rows * batches * H * V)) continue;
                    const float o = R.out_scale * fmaf(e, inter[r][q], intra[r][q]);
                    if (R.out_f32) ((float*)R.out)[at + q] = o;
                    else ((T*)R.out)[at + q] = from_f32<T>(o);
                }
            }
            __syncthreads();  // every read of H before its update
        }
        const float2 dec = n - 1 + off == kC ? full : decay_power(la, n - 1 + off);
        for (int e = tid; e < kC * L.K4; e += kThreads) {
            const int j = e / L.K4, k = e - j * L.K4;
            if (j < n) sK[j * L.ldk + k] *= sTab[R.reverse ? j : n - 1 - j];
        }
        __syncthreads();
        for (int kb = 4 * rg; kb < L.K4; kb += 64) {
            float acc[4][4] = {};
#pragma unroll 4
            for (int j = 0; j < kC; ++j) {
                const float4 a = *reinterpret_cast<const float4*>(sK + j * L.ldk + kb);
                const float4 b = *reinterpret_cast<const float4*>(sV + j * kVT + cg);
                const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc[r][0] = fmaf(av[r], b.x, acc[r][0]);
                    acc[r][1] = fmaf(av[r], b.y, acc[r][1]);
                    acc[r][2] = fmaf(av[r], b.z, acc[r][2]);
                    acc[r][3] = fmaf(av[r], b.w, acc[r][3]);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float4* hp = reinterpret_cast<float4*>(sH + (kb + r) * kVT + cg);
                float4 h = *hp;
                h.x = fmaf(h.x, dec.x, fmaf(h.x, dec.y, acc[r][0]));
                h.y = fmaf(h.y, dec.x, fmaf(h.y, dec.y, acc[r][1]));
                h.z = fmaf(h.z, dec.x, fmaf(h.z, dec.y, acc[r][2]));
                h.w = fmaf(h.w, dec.x, fmaf(h.w, dec.y, acc[r][3]));
                *hp = h;
            }
        }
        off = 1;
    }
    __syncthreads();
    float* dst = nullptr;
    float mul = 1.f;
    if (!kOut) {
        dst = p.states + it.slot * K * V;
    } else if (R.fin && it.seg == it.nseg - 1) {
        dst = R.fin + chain * K * V;
        mul = R.fin_scale * (R.reverse && it.len > 0 ? decay_power(la, 1).x : 1.f);
    }
    if (dst) {
        const long long extent = kOut ? chains * K * V : p.plan.slots() * K * V;
        const float* dst0 = kOut ? R.fin : p.states;
        (void)extent, (void)dst0;
        for (int e = tid; e < K * kVT; e += kThreads) {
            const int k = e / kVT, c = e % kVT;
            if (c < vn && SSD_INB(dst - dst0 + (long long)k * V + v0 + c, extent)) dst[(long long)k * V + v0 + c] = sH[e] * mul;
        }
    }
}

// The state entering each item of a cut chain, in place: slot i holds what item
// i builds from zero and becomes the state after it,
//     e <- l^(tokens of item i) e + slot_i,
// e starting as the chain's initial state.  `tiles` blocks per chain, a thread
// per state element at a time; the work is one pass over the slots.
__global__ void __launch_bounds__(256) scan_combine_kernel(const ScanLaunch p, int tiles) {
    __shared__ ScanItem sItem;
    next_may_start();
    const long long cr = blockIdx.x / tiles;  // chain and role
    if (threadIdx.x < 32) {
        const ScanItem f = scan_item(p.plan, p.plan.packed ? cr : p.plan.nfull + cr * p.plan.nseg);
        if (threadIdx.x == 0) sItem = f;
    }
    __syncthreads();
    const ScanItem it = sItem;
    if (!it.valid || it.nseg < 2 || it.seg > 0) {  // (packed: not a first item's number)
        if (blockIdx.x == 0) wait_for_earlier();
        return;
    }
    const ScanRole& R = p.role[it.role];
    const int K = R.K, V = R.V;
    const float la = p.decay[it.head];
    const long long step = p.plan.packed ? (long long)p.plan.H * p.plan.nroles : 1;
    const long long chain = (long long)it.seq * p.plan.H + it.head;
    const float2 whole = decay_power(la, p.plan.seg_tokens);
    // the first item of a backward scan is the sequence's last, shorter piece,
    // and its initial state meets the last token undecayed
    const int n0 = R.reverse ? it.len - (it.nseg - 1) * p.plan.seg_tokens - 1 : p.plan.seg_tokens;
    const float2 first = decay_power(la, n0);
    wait_for_earlier();
    // four elements at a time: their loads are on the way together
    constexpr int U = 4;
    const int apart = tiles * 256, KV = K * V;
    for (int e0 = (blockIdx.x % tiles) * 256 + threadIdx.x; e0 < KV; e0 += U * apart) {
        float h[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * apart;
            h[u] = 0.f;
            if (R.init && e < KV) {
                const long long at = chain * KV + (e / V) * R.init_k + (e % V) * R.init_v;
                if (SSD_INB(at, (long long)p.plan.B * p.plan.H * KV)) h[u] = R.init[at] * R.init_scale;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * apart;
            const long long at = it.slot_init * KV + e;
            if (R.init && e < KV && SSD_INB(at, p.plan.slots() * KV)) p.states[at] = h[u];
        }
        // a slot's numbers are on their way while the one before is worked on
        float* at = p.states + it.slot * KV + e0;
        const long long next = step * KV;
        float z[U];
        auto fetch = [&](const float* from) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                z[u] = e0 + u * apart < KV && SSD_INB(from - p.states + u * apart, p.plan.slots() * KV) ? from[u * apart] : 0.f;
        };
        fetch(at);
        for (int i = 0; i + 1 < it.nseg; ++i, at += next) {
            const float2 d = i == 0 ? first : whole;
#pragma unroll
            for (int u = 0; u < U; ++u) h[u] = fmaf(h[u], d.x, fmaf(h[u], d.y, z[u]));
            if (i + 2 < it.nseg) fetch(at + next);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e0 + u * apart < KV && SSD_INB(at - p.states + u * apart, p.plan.slots() * KV)) at[u * apart] = h[u];
        }
    }
}

// out[row][g][d] = sum over the heads h of the group of part[row][h][d], in the order
// of the heads, for the rows of some sequence; VEC numbers a thread, `across`
// threads along a row (a power of two).
template <typename T, int VEC>
__global__ void __launch_bounds__(256) group_sum_kernel(const float* part, T* out, long long rows, int D,
                                                        int G, int share, const int* cu, int B, int across) {
    next_may_start();
    wait_for_earlier();
    const int x = threadIdx.x % across, y = threadIdx.x / across, per = 256 / across;
    const int units = G * D / VEC, per_group = D / VEC;
    long long lo = 0, hi = rows;
    if (cu) {  // (packed rows number less than 2^31)
        lo = min(max(cu[0], 0), (int)rows);
        hi = min(max(cu[B], 0), (int)rows);
    }
    for (long long r = lo + (long long)blockIdx.x * per + y; r < hi; r += (long long)gridDim.x * per)
        for (int u = x; u < units; u += across) {
            const int g = u / per_group, d = (u - g * per_group) * VEC;
            const long long from = ((r * G + g) * share) * D + d, to = (r * G + g) * D + d;
            float s[VEC] = {};
            for (int h = 0; h < share; ++h) {
                if (!SSD_INB(from + (long long)h * D + VEC - 1, rows * G * share * D)) continue;
                if constexpr (VEC == 4) {
                    const float4 f = __ldcg(reinterpret_cast<const float4*>(part + from + (long long)h * D));
                    s[0] += f.x;
                    s[1] += f.y;
                    s[2] += f.z;
                    s[3] += f.w;
                } else {
                    s[0] += __ldcg(part + from + (long long)h * D);
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (SSD_INB(to + i, rows * G * D)) out[to + i] = from_f32<T>(s[i]);
        }
}

}  // namespace

cudaError_t launch_scan_simt(const ScanLaunch& s, bool state_only, cudaStream_t st) {
    int V = 1, K = 1;
    for (int r = 0; r < s.plan.nroles; ++r) {
        V = s.role[r].V > V ? s.role[r].V : V;
        K = s.role[r].K > K ? s.role[r].K : K;
    }
    const int ntiles = (V + kVT - 1) / kVT;
    const long long grid = (state_only ? s.plan.state_items() : s.plan.items) * ntiles;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const size_t smem = simt_layout(K).bytes;
    auto kernel = s.bf16 ? (state_only ? scan_simt_kernel<__nv_bfloat16, false> : scan_simt_kernel<__nv_bfloat16, true>)
                         : (state_only ? scan_simt_kernel<float, false> : scan_simt_kernel<float, true>);
    cudaError_t e = allow_smem(kernel, 1024);
    if (e != cudaSuccess) return e;
    return launch_in_call(kernel, (unsigned)grid, kThreads, smem, st, !s.reset, s, ntiles);
}

cudaError_t launch_scan_combine(const ScanLaunch& s, cudaStream_t st) {
    int KV = 1;
    for (int r = 0; r < s.plan.nroles; ++r) KV = s.role[r].K * s.role[r].V > KV ? s.role[r].K * s.role[r].V : KV;
    // enough blocks to fill the GPU, none more
    const long long chains = s.plan.cut_chains();
    int tiles = (KV + 1023) / 1024;  // (four elements a thread)
    while (tiles > 1 && chains * tiles > 148 * 8) tiles = (tiles + 1) / 2;
    const long long grid = chains * tiles;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_in_call(scan_combine_kernel, (unsigned)grid, 256, 0, st, true, s, tiles);
}

cudaError_t launch_group_sum(const float* part, void* out, long long rows, int H, int G, int D, const int* cu, int B,
                             bool bf16, cudaStream_t st) {
    const int vec = D % 4 == 0 ? 4 : 1;
    const long long units = (long long)G * D / vec;
    int across = 1;
    while (across < 256 && across < units) across *= 2;
    const long long want = (rows + 256 / across - 1) / (256 / across);
    const unsigned grid = (unsigned)(want < 148 * 16 ? want : 148 * 16);
    auto run = [&](auto kernel, auto to) {
        return launch_in_call(kernel, grid, 256, 0, st, true, part, to, rows, D, G, H / G, cu, B, across);
    };
    auto* b = (__nv_bfloat16*)out;
    auto* f = (float*)out;
    if (bf16) return vec == 4 ? run(group_sum_kernel<__nv_bfloat16, 4>, b) : run(group_sum_kernel<__nv_bfloat16, 1>, b);
    return vec == 4 ? run(group_sum_kernel<float, 4>, f) : run(group_sum_kernel<float, 1>, f);
}

}  // namespace ssd

// linear_tc.cu -- the linear-attention scan on the fifth-generation tensor
// cores (bf16, K and V up to 128, padded with zeros to 64 or 128).
//
// One block per item (a chain or a piece of one), chunks of 128 tokens in scan
// order.  With positions i, j in a chunk of n tokens, l = exp(decay) and H the
// fp32 state entering it:
//     S   = Q K^T                                   scores
//     P   = S o L,  L_ij = l^|i-j| on the causal side, else 0    (bf16, in TMEM)
//     out = out_scale (P V + diag(l^(i+1)) Q H)     two accumulators, joined in fp32
//     Z   = (w o K)^T V,  w_j = l^(n-1-j)           the chunk's own state
//     H  <- l^n H + Z                               in registers, fp32
// and the mirror image for a scan backwards.  No factor exceeds 1: L is built
// from two factors <= 1 per 32 x 32 block, one table of powers made in 64 bits.
//
// Precision.  P, and H as an operand, are rounded to bf16 (their errors are
// those of the result's own rounding).  The state itself is fp32 and outlives
// the call, so w o K must not lose bits: it enters the product as kPieces bf16
// numbers whose sum is the fp32 product: 3 leave an error below 2^-24 and are
// used where the state is a result, 2 (below 2^-17) where it only enters
// outputs.  l^n multiplies H at every chunk and is kept as a sum of two fp32
// numbers, or its rounding would grow with the number of chunks.
//
// Warp roles (608 threads):
//   0-3    scores -> P (thread = row i)
//   4-7    w o K: the first piece in K's own place in shared memory once the
//          scores are done, the others in two buffers of 32 tokens in turn;
//          rows behind a partial chunk's end become zeros there, in V too (with
//          packed sequences they hold the next sequence's tokens)
//   8-15   state and output (two warps per TMEM lane quadrant)
//   16     TMA loads; 17  TMEM, MMA issue
//   18     TMA stores: the output tile takes the place of the chunk's K in shared
//          memory (plain stores of rows by their threads touch 32 lines each: they
//          kept the load/store unit busy for 2000 of a chunk's cycles)
// MMA order per chunk: S, Q H, half of Z, P V, the other half of Z, so that the
// next chunk's S finds P consumed and the conversions run beside other products.
//
// With V = 128 the lanes of Z are the state's columns (v), else its rows (k): an
// MMA takes 128 rows, and the other order would waste half of them.
#include "../common.cuh"
#include "../debug_checks.cuh"
#include "../linear.h"
#include "../tc_common.cuh"
#include "../tmap.h"

namespace ssd {
namespace {

constexpr int kBlk = kScanChunk;         // 128 tokens: the MMA's M
constexpr int kThreads = 608;
constexpr uint32_t kPanel = kBlk * 128;  // 128 rows of 64 bf16
constexpr uint32_t kPart = 32 * 128;     // 32 rows of 64 bf16

// TMEM columns
constexpr uint32_t COL_S = 0;    // scores, then P in the first 64
constexpr uint32_t COL_O1 = 128;
constexpr uint32_t COL_O2 = 256;
constexpr uint32_t COL_Z = 384;

constexpr int kMaxBufs = 12;
struct __align__(8) Bars {
    uint64_t full[kMaxBufs], empty[kMaxBufs];
    uint64_t s_full, p_full, o_full, o_free;
    uint64_t kt_full[2], kt_free[2];
    uint64_t z_full, z_free, h_full, h_free, staged;
    uint64_t done;
};

struct TcParams {
    CUtensorMap map[kScanRoles][4];  // q, k, v, out
    ScanLaunch s;
};

// Shared memory of a variant.  K = V = 128: a ring of five tiles in the order
// q, k, v, q, ... (a whole second chunk does not fit); else whole chunks.
template <int KP, int VP, int kPieces>
struct Layout {
    static constexpr bool kRing = KP == 128 && VP == 128;
    static constexpr uint32_t kKB = KP / 64 * kPanel, kVB = VP / 64 * kPanel;
    static constexpr uint32_t kChunk = 2 * kKB + kVB;
    static constexpr int kStages = kRing ? 0 : KP == 128 ? 2 : VP == 128 ? 3 : 4;
    static constexpr int kBufs = kRing ? 5 : 3 * kStages;
    static constexpr uint32_t OFF_PART = kRing ? 5 * 2 * kPanel : kStages * kChunk;
    static constexpr uint32_t kPartB = KP / 64 * kPart;  // one piece of 32 tokens
    static constexpr uint32_t OFF_H = OFF_PART + 2 * (kPieces - 1) * kPartB;
    static constexpr uint32_t OFF_TAB = OFF_H + (uint32_t)KP * VP * 2;
    static constexpr uint32_t OFF_REV = OFF_TAB + 164 * 4;
    static constexpr uint32_t OFF_BAR = OFF_REV + 160 * 4;
    static constexpr uint32_t OFF_MISC = OFF_BAR + (sizeof(Bars) + 15) / 16 * 16;
    static constexpr uint32_t OFF_ITEM = OFF_MISC + 16;
    static constexpr size_t kBytes = 1024 + OFF_ITEM + sizeof(ScanItem);
    static_assert(kBytes <= 232448, "shared memory above the 227 KB per-block limit");

    // buffer, its use count and its place, of tile `which` (0 q, 1 k, 2 v) of chunk c;
    // a state-only scan loads no q
    struct Buf { uint32_t i, use, off; };
    static __device__ __forceinline__ Buf buf(uint32_t c, uint32_t which, bool out) {
        Buf b;
        if (kRing) {
            const uint32_t n = out ? 3 * c + which : 2 * c + which - 1;
            b.use = n / 5;
            b.i = n - 5 * b.use;
            b.off = b.i * 2 * kPanel;
        } else {
            b.use = c / (uint32_t)(kStages ? kStages : 1);
            const uint32_t st = c - b.use * kStages;
            b.i = 3 * st + which;
            b.off = st * kChunk + (which > 0 ? kKB : 0) + (which > 1 ? kKB : 0);
        }
        return b;
    }
};

template <int KP, int VP, bool kOut, int kPieces>
__global__ void __launch_bounds__(kThreads, 1) scan_tc_kernel(const __grid_constant__ TcParams p) {
    using L = Layout<KP, VP, kPieces>;
    constexpr bool kLaneV = VP == 128;         // lanes of Z: v, else k
    constexpr int CH = kLaneV ? KP / 2 : 32;   // state columns of a thread
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sPart = sm + L::OFF_PART;  // [2][kPieces - 1] pieces of 32 tokens
    uint8_t* sH = sm + L::OFF_H;
    float* sTab = reinterpret_cast<float*>(sm + L::OFF_TAB) + 32;  // l^0 .. l^128; l^d = 0 for -32 <= d < 0
    float* sRev = reinterpret_cast<float*>(sm + L::OFF_REV);       // l^127 .. l^0, then zeros for d = -1 .. -32
    Bars* bars = reinterpret_cast<Bars*>(sm + L::OFF_BAR);
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + L::OFF_MISC);
    int* sAbort = reinterpret_cast<int*>(sm + L::OFF_MISC + 4);
    ScanItem* sItem = reinterpret_cast<ScanItem*>(sm + L::OFF_ITEM);
    volatile int* abort_v = sAbort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (p.s.reset && blockIdx.x == 0 && threadIdx.x == 0) *p.s.status = kDevOk;
    if (warp == 0) {
        ScanItem f = scan_item(p.s.plan, blockIdx.x);
        if (f.valid) scan_item_tokens(f, p.s.plan.seg_tokens, p.s.role[f.role].reverse);
        if (lane == 0) *sItem = f;
    }
    __syncthreads();
    const ScanItem it = *sItem;
    if (!it.valid || (!kOut && it.seg == it.nseg - 1)) return;
    const ScanRole& R = p.s.role[it.role];
    const int K = R.K, V = R.V;
    const bool rev = R.reverse != 0;
    const float la = p.s.decay[it.head];
    const int H = p.s.plan.H;
    const long long chain = (long long)it.seq * H + it.head;
    const long long chains = (long long)p.s.plan.B * H;
    (void)chains;
    const int span = it.t1 - it.t0;
    const int nch = (span + kBlk - 1) / kBlk;

    if (threadIdx.x == 32) {
        for (int i = 0; i < L::kBufs; ++i) {
            tc::mbar_init(&bars->full[i], 1);
            tc::mbar_init(&bars->empty[i], 1);
        }
        tc::mbar_init(&bars->s_full, 1);
        tc::mbar_init(&bars->p_full, 4);
        tc::mbar_init(&bars->o_full, 1);
        tc::mbar_init(&bars->o_free, 8);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars->kt_full[i], 4);
            tc::mbar_init(&bars->kt_free[i], 1);
        }
        tc::mbar_init(&bars->z_full, 1);
        tc::mbar_init(&bars->z_free, 8);
        tc::mbar_init(&bars->h_full, 8);
        tc::mbar_init(&bars->h_free, 1);
        tc::mbar_init(&bars->staged, 8);
        tc::mbar_init(&bars->done, 1);
        *sAbort = 0;
        tc::fence_mbar_init();
    }
    if (warp == 17) {
        tc::tmem_alloc(sTmem, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x >= 64 && threadIdx.x - 64 <= kBlk + 32) {
        const int d = (int)threadIdx.x - 96;
        const float e = d < 0 ? 0.f : decay_power(la, d).x;
        sTab[d] = e;
        if (d < kBlk) sRev[kBlk - 1 - d] = e;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *sTmem;

    auto fail = [&]() {
        *reinterpret_cast<volatile int*>(sAbort) = 1;
        atomicExch(p.s.status, kDevTimeout);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return tc::mbar_wait(bar, parity, abort_v); };
    // the same decision in every lane: what follows is executed by whole warps
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_v));
    };
    // first token (in the sequence) and tokens of the c-th chunk in scan order
    auto chunk_at = [&](int c) -> int { return it.t0 + (rev ? nch - 1 - c : c) * kBlk; };
    auto chunk_n = [&](int t) -> int { return min(kBlk, it.t1 - t); };
    // a chunk of n tokens whose output leaves by plain stores: fp32, or a packed
    // sequence's end, behind which the rows are another's
    auto direct = [&](int n) -> bool { return R.out_f32 || (p.s.plan.packed && n < kBlk); };

    if (warp == 16) {
        if (lane == 0) {
            // ------------------------------------------------- TMA loads ----
            bool ok = true;
            const int head[3] = {it.head / R.q.share, it.head / R.k.share, it.head / R.v.share};
            int c = 0;
            for (; ok && c < nch; ++c) {
                const int row = (int)(it.row0 + chunk_at(c));
#pragma unroll
                for (int w = kOut ? 0 : 1; w < 3; ++w) {
                    const auto b = L::buf(c, w, kOut);
                    if (b.use > 0 && !wait(&bars->empty[b.i], (b.use - 1) & 1)) { ok = false; break; }
                    const int panels = (w == 2 ? VP : KP) / 64;
                    tc::mbar_arrive_expect_tx(&bars->full[b.i], panels * kPanel);
                    for (int x = 0; x < panels; ++x)
                        tc::tma_load_4d(sm + b.off + x * kPanel, &p.map[it.role][w], &bars->full[b.i], 64 * x,
                                        head[w], row, it.batch);
                }
            }
            if (!ok) {
                fail();
                // no copy may still be landing in shared memory when the block exits
                for (int cc = c > 4 ? c - 4 : 0; cc < c; ++cc)
                    for (int w = kOut ? 0 : 1; w < 3; ++w) {
                        const auto b = L::buf(cc, w, kOut);
                        tc::mbar_wait(&bars->full[b.i], b.use & 1, nullptr, 200000000ull);
                    }
            }
        }
    } else if (warp == 17) {
        // ----------------------------------------------------- MMA issue ----
        constexpr uint32_t id_s = tc::idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint32_t id_pv = tc::idesc_bf16_f32(128, VP, 0, 1);
        constexpr uint32_t id_qh = tc::idesc_bf16_f32(128, VP, 0, kLaneV ? 0 : 1);
        constexpr uint32_t id_z = tc::idesc_bf16_f32(128, kLaneV ? KP : VP, 1, 1);
        const uint32_t base = __shfl_sync(0xffffffffu, tc::smem_u32(sm), 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const int chunks = __shfl_sync(0xffffffffu, nch, 0);
        const uint64_t kmaj = tc::smem_desc_sw128(base, 16, 1024);       // rows contiguous along the contraction
        const uint64_t mnmaj = tc::smem_desc_sw128(base, kPanel, 1024);  // contraction along the rows
        const uint64_t partmn = tc::smem_desc_sw128(base + L::OFF_PART, kPart, 1024);
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint32_t ph = c & 1, was = (c - 1) & 1;
            const auto bk = L::buf(c, 1, kOut), bv = L::buf(c, 2, kOut);
            const uint64_t dkk = tc::desc_adv(kmaj, bk.off), dkm = tc::desc_adv(mnmaj, bk.off), dvm = tc::desc_adv(mnmaj, bv.off);
            if (kOut) {
                const auto bq = L::buf(c, 0, kOut);
                const uint64_t dq = tc::desc_adv(kmaj, bq.off);
                // the scores overwrite the P that the last P V read
                ok = wait_warp(&bars->full[bq.i], bq.use & 1) && wait_warp(&bars->full[bk.i], bk.use & 1) &&
                     (c == 0 || wait_warp(&bars->o_full, was));
                if (!ok) break;
                tc::tc_fence_after();
                if (tc::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < KP / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kPanel + (kk & 3) * 32;
                        tc::mma_ss(tm + COL_S, tc::desc_adv(dq, off), tc::desc_adv(dkk, off), id_s, kk > 0);
                    }
                    tc::mma_commit(&bars->s_full);
                }
                __syncwarp();
                ok = wait_warp(&bars->h_full, ph) && (c == 0 || wait_warp(&bars->o_free, was));
                if (!ok) break;
                tc::tc_fence_after();
                if (tc::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < KP / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kPanel + (kk & 3) * 32;
                        const uint64_t dh = kLaneV ? tc::desc_adv(kmaj, L::OFF_H + off) : tc::desc_adv(mnmaj, L::OFF_H + kk * 2048);
                        tc::mma_ss(tm + COL_O2, tc::desc_adv(dq, off), dh, id_qh, kk > 0);
                    }
                    tc::mma_commit(&bars->h_free);
                    tc::mma_commit(&bars->empty[bq.i]);
                }
                __syncwarp();
            }
            ok = wait_warp(&bars->full[bv.i], bv.use & 1) && (c == 0 || wait_warp(&bars->z_free, was));
            if (!ok) break;
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                // Z (+)= (w o K)^T V over the 32 tokens of quarter u
                const uint32_t qn = 4u * c + u, s = qn & 1;
                ok = wait_warp(&bars->kt_full[s], (qn >> 1) & 1);
                if (!ok) break;
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    const uint64_t dv = tc::desc_adv(dvm, u * 4096);
                    const uint64_t dk = tc::desc_adv(dkm, u * 4096);
                    const uint64_t dp = tc::desc_adv(partmn, s * (kPieces - 1) * L::kPartB);
#pragma unroll
                    for (int x = 0; x < kPieces; ++x) {
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            const uint64_t a = x == 0 ? tc::desc_adv(dk, kk * 2048)
                                                      : tc::desc_adv(dp, (x - 1) * L::kPartB + kk * 2048);
                            const uint64_t b = tc::desc_adv(dv, kk * 2048);
                            tc::mma_ss(tm + COL_Z, kLaneV ? b : a, kLaneV ? a : b, id_z, (u > 0 || x > 0 || kk > 0) ? 1u : 0u);
                        }
                    }
                    tc::mma_commit(&bars->kt_free[s]);
                }
                __syncwarp();
                if (kOut && u == 1) {
                    ok = wait_warp(&bars->p_full, ph);
                    if (!ok) break;
                    tc::tc_fence_after();
                    if (tc::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kBlk / 16; ++kk)
                            tc::mma_ts(tm + COL_O1, tm + COL_S + kk * 8, tc::desc_adv(dvm, kk * 2048), id_pv, kk > 0);
                        tc::mma_commit(&bars->o_full);
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (tc::elect_one()) {
                tc::mma_commit(&bars->z_full);
                if (!kOut) tc::mma_commit(&bars->empty[bk.i]);  // else the output leaves through it first
                tc::mma_commit(&bars->empty[bv.i]);
            }
            __syncwarp();
        }
        if (!ok) fail();
        // every product issued must be complete before TMEM is released
        if (tc::elect_one()) tc::mma_commit(&bars->done);
        __syncwarp();
        tc::mbar_wait(&bars->done, 0, nullptr, 200000000ull);
    } else if (warp == 18) {
        if (kOut && lane == 0) {
            // -------------------------------- the output tile, from K's place ----
            bool ok = true;
            for (int c = 0; c < nch; ++c) {
                const int t = chunk_at(c), n = chunk_n(t);
                const auto bk = L::buf(c, 1, kOut);
                ok = wait(&bars->staged, c & 1);
                if (!ok) break;
                if (!direct(n)) {
                    for (int x = 0; x < VP / 64; ++x)
                        if (64 * x < V)
                            tc::tma_store_4d(&p.map[it.role][3], sm + bk.off + x * kPanel, 64 * x, it.head,
                                             (int)(it.row0 + t), it.batch);
                    tc::bulk_commit();
                    tc::bulk_wait_read<0>();
                }
                tc::mbar_arrive(&bars->empty[bk.i]);
            }
            if (!ok) fail();
        }
    } else if (warp < 4) {
        if (kOut) {
            // ------------------------------------- P = S o L, thread = row ----
            const uint32_t ts = tmem + ((uint32_t)(warp * 32) << 16) + COL_S;
            // l^|i-j| of row i against the columns of block jb: 32 consecutive
            // entries of a table, neighbouring lanes one apart
            const float* near = rev ? sTab - (32 * warp + lane) : sRev + kBlk - 1 - (32 * warp + lane);
            const uint32_t diag = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
            bool ok = true;
#pragma unroll 1
            for (int c = 0; c < nch; ++c) {
                const int n = chunk_n(chunk_at(c));
                ok = wait_warp(&bars->s_full, c & 1);
                if (!ok) break;
                tc::tc_fence_after();
#pragma unroll 1
                for (int jb = 0; jb < 4; ++jb) {
                    // the block's columns on the causal side and in the chunk
                    uint32_t m = jb == warp ? diag : (rev ? jb > warp : jb < warp) ? 0xffffffffu : 0u;
                    if (n < 32 * jb + 32) m &= n > 32 * jb ? 0xffffffffu >> (32 * jb + 32 - n) : 0u;
                    uint32_t r[16];
                    if (__any_sync(0xffffffffu, m != 0)) {
                        float s[32];
                        tc::tmem_ld32(ts + 32 * jb, s);
                        const float* w = near + 32 * jb;
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 v = tc::mul2(make_float2(s[2 * j], s[2 * j + 1]), make_float2(w[2 * j], w[2 * j + 1]));
                            s[2 * j] = v.x;
                            s[2 * j + 1] = v.y;
                        }
                        // a product with 0 would keep a NaN of a masked place
                        if (!__all_sync(0xffffffffu, m == 0xffffffffu)) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) s[j] = (m >> j) & 1 ? s[j] : 0.f;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) r[j] = tc::pack_bf16x2(s[2 * j], s[2 * j + 1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) r[j] = 0;
                    }
                    // columns 16 jb .. overlay scores of blocks that are read
                    tc::tmem_st16(ts + 16 * jb, r);
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars->p_full);
            }
            if (!ok) fail();
        }
    } else if (warp < 8) {
        // ------------------------------------------------ w o K in pieces ----
        const int t = threadIdx.x - 128;
        bool ok = true;
#pragma unroll 1
        for (int c = 0; ok && c < nch; ++c) {
            const int n = chunk_n(chunk_at(c));
            const auto bk = L::buf(c, 1, kOut), bv = L::buf(c, 2, kOut);
            ok = wait_warp(&bars->full[bk.i], bk.use & 1) && (!kOut || wait_warp(&bars->s_full, c & 1));
            if (!ok) break;
            if (n < kBlk) {
                ok = wait_warp(&bars->full[bv.i], bv.use & 1);
                if (!ok) break;
                for (int e = t; e < (kBlk - n) * 8 * (VP / 64); e += 128) {
                    const int x = e / ((kBlk - n) * 8), f = e - x * (kBlk - n) * 8;
                    *reinterpret_cast<uint4*>(sm + bv.off + x * kPanel + (n + f / 8) * 128 + (f & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                const uint32_t qn = 4u * c + u, s = qn & 1;
                if (qn >= 2) {
                    ok = wait_warp(&bars->kt_free[s], ((qn >> 1) - 1) & 1);
                    if (!ok) break;
                }
                const int row = 32 * u + lane;
                const bool in = row < n;
                const float w = in ? sTab[rev ? row : n - 1 - row] : 0.f;
                const float2 w2 = make_float2(w, w), minus = make_float2(-1.f, -1.f);
                uint8_t* krow = sm + bk.off + row * 128;
                uint8_t* prow = sPart + s * (kPieces - 1) * L::kPartB + lane * 128;
#pragma unroll 1
                for (int x = 0; x < KP / 64; ++x) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // eight neighbouring rows take eight different 16-byte columns
                        const int cc = ((2 * (warp - 4) + i) ^ (row & 7)) * 16;
                        const uint4 kv = *reinterpret_cast<const uint4*>(krow + x * kPanel + cc);
                        const uint32_t in4[4] = {kv.x, kv.y, kv.z, kv.w};
                        uint32_t o[kPieces][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 f = tc::mul2(tc::unpack_bf16x2(in4[e]), w2);
#pragma unroll
                            for (int q = 0; q < kPieces; ++q) {
                                o[q][e] = in ? tc::pack_bf16x2(f.x, f.y) : 0u;
                                if (q + 1 < kPieces) f = tc::fma2(tc::unpack_bf16x2(o[q][e]), minus, f);
                            }
                        }
                        *reinterpret_cast<uint4*>(krow + x * kPanel + cc) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
#pragma unroll
                        for (int q = 1; q < kPieces; ++q)
                            *reinterpret_cast<uint4*>(prow + (q - 1) * L::kPartB + x * kPart + cc) =
                                make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars->kt_full[s]);
            }
        }
        if (!ok) fail();
    } else if (warp < 16) {
        // ------------------------------------------------ state and output ----
        const int quad = warp & 3, half = (warp - 8) >> 2;
        const int lr = quad * 32 + lane;  // lane of TMEM
        const int c0 = half * CH;
        const bool holds = kLaneV || lr < KP;  // K = 64: lanes behind it hold nothing
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        float h[CH];
        const bool from_init = it.seg == 0;
        // element of column c: (k, v)
        auto k_of = [&](int c) -> int { return kLaneV ? c0 + c : lr; };
        auto v_of = [&](int c) -> int { return kLaneV ? lr : c0 + c; };
#pragma unroll
        for (int c = 0; c < CH; ++c) h[c] = 0.f;
        if (kOut && holds && (!from_init || R.init)) {
            const float* src = from_init ? R.init + chain * K * V : p.s.states + it.slot_prev * K * V;
            const long long sk = from_init ? R.init_k : V, sv = from_init ? R.init_v : 1;
            const float mul = from_init ? R.init_scale : 1.f;
            src += k_of(0) * sk + v_of(0) * sv;
            const long long step = kLaneV ? sk : sv;
            const int have = kLaneV ? (lr < V ? K - c0 : 0) : (lr < K ? V - c0 : 0);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (c < have && SSD_INB(k_of(c) * sk + v_of(c) * sv, (long long)K * V)) h[c] = *src * mul;
                src += step;
            }
        }
        // H as an operand: [v][k] (lanes v) or [k][v]
        auto put_h = [&]() {
            if (holds) {
                uint8_t* row = sH + (CH == 64 ? half * kPanel : 0) + lr * 128;
                const int first = CH == 64 ? 0 : half * 4;
#pragma unroll
                for (int x = 0; x < CH / 8; ++x)
                    *reinterpret_cast<uint4*>(row + (((first + x) ^ (lr & 7)) << 4)) =
                        make_uint4(tc::pack_bf16x2(h[8 * x], h[8 * x + 1]), tc::pack_bf16x2(h[8 * x + 2], h[8 * x + 3]),
                                   tc::pack_bf16x2(h[8 * x + 4], h[8 * x + 5]), tc::pack_bf16x2(h[8 * x + 6], h[8 * x + 7]));
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars->h_full);
        };
        if (kOut && nch > 0) put_h();
        // a backward scan's initial state meets its first token undecayed
        int off = from_init && rev ? 0 : 1;
        const float2 whole = decay_power(la, kBlk);
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            const int t = chunk_at(c), n = chunk_n(t);
            ok = wait_warp(&bars->z_full, c & 1);
            if (!ok) break;
            tc::tc_fence_after();
            const float2 dec = n - 1 + off == kBlk ? whole : decay_power(la, n - 1 + off);
            const float2 dx = make_float2(dec.x, dec.x), dy = make_float2(dec.y, dec.y);
#pragma unroll
            for (int x = 0; x < CH / 32; ++x) {
                float z[32];
                tc::tmem_ld32(tl + COL_Z + c0 + 32 * x, z);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 o = make_float2(h[32 * x + e], h[32 * x + e + 1]);
                    const float2 w = tc::fma2(o, dx, tc::fma2(o, dy, make_float2(z[e], z[e + 1])));
                    h[32 * x + e] = w.x;
                    h[32 * x + e + 1] = w.y;
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars->z_free);
            if (kOut) {
                if (c + 1 < nch) {
                    ok = wait_warp(&bars->h_free, c & 1);  // Q H has read this chunk's H
                    if (!ok) break;
                    put_h();
                }
                ok = wait_warp(&bars->o_full, c & 1);
                if (!ok) break;
                tc::tc_fence_after();
                const float e = lr < n ? sTab[(rev ? n - 1 - lr : lr) + off] * R.out_scale : 0.f;
                const long long row = (long long)it.batch * p.s.plan.T + it.row0 + t + lr;
                const long long at0 = (row * H + it.head) * V;
                const bool plain = direct(n);
                uint8_t* tile = sm + L::buf(c, 1, kOut).off + lr * 128;  // this chunk's K is consumed (z_full)
#pragma unroll 1
                for (int x = 0; x < VP / 32; ++x) {
                    const int col = half * (VP / 2) + 16 * x;
                    float a[16], b[16];
                    tc::tmem_ld16(tl + COL_O1 + col, a);
                    tc::tmem_ld16(tl + COL_O2 + col, b);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 16; ++q) a[q] = fmaf(e, b[q], R.out_scale * a[q]);
                    uint32_t o[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) o[q] = tc::pack_bf16x2(a[2 * q], a[2 * q + 1]);
                    if (!plain) {
                        const int cc = (col & 63) >> 3;
                        uint8_t* d = tile + (col >> 6) * kPanel;
                        *reinterpret_cast<uint4*>(d + ((cc ^ (lr & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(d + (((cc + 1) ^ (lr & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                    } else {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int cy = col + 8 * y;
                            if (lr >= n || cy >= V ||
                                !SSD_INB(at0 + cy + 7, (p.s.plan.packed ? 1LL : p.s.plan.B) * p.s.plan.T * H * V))
                                continue;
                            if (R.out_f32) {
                                float4* f = reinterpret_cast<float4*>((float*)R.out + at0 + cy);
                                f[0] = make_float4(a[8 * y], a[8 * y + 1], a[8 * y + 2], a[8 * y + 3]);
                                f[1] = make_float4(a[8 * y + 4], a[8 * y + 5], a[8 * y + 6], a[8 * y + 7]);
                            } else {
                                *reinterpret_cast<uint4*>((__nv_bfloat16*)R.out + at0 + cy) =
                                    make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                            }
                        }
                    }
                }
                tc::tc_fence_before();
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&bars->o_free);
                    tc::mbar_arrive(&bars->staged);
                }
            }
            off = 1;
        }
        if (!ok) fail();
        // the state after the item
        float* dst = nullptr;
        float mul = 1.f;
        if (!kOut) {
            dst = p.s.states + it.slot * K * V;
        } else if (R.fin && it.seg == it.nseg - 1) {
            dst = R.fin + chain * K * V;
            mul = R.fin_scale * (rev && it.len > 0 ? decay_power(la, 1).x : 1.f);
        }
        if (ok && dst && holds && SSD_INB(kOut ? chain : it.slot, kOut ? chains : p.s.plan.slots())) {
            dst += (long long)k_of(0) * V + v_of(0);
            const int step = kLaneV ? V : 1;
            const int have = kLaneV ? (lr < V ? K - c0 : 0) : (lr < K ? V - c0 : 0);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (c < have) *dst = h[c] * mul;
                dst += step;
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        __syncwarp();
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

int padded(int d) { return d <= 64 ? 64 : 128; }

cudaError_t role_maps(const ScanRole& r, const ScanPlan& p, CUtensorMap* m) {
    const RowTensor* t[3] = {&r.q, &r.k, &r.v};
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 3 && e == cudaSuccess; ++i)
        e = make_tmap_bf16_rows(&m[i], t[i]->p, i == 2 ? r.V : r.K, p.H / t[i]->share, p.T, p.packed ? 1 : p.B,
                                t[i]->head, t[i]->token, t[i]->batch, kBlk);
    if (e == cudaSuccess && !r.out_f32)
        e = make_tmap_bf16_rows(&m[3], r.out, r.V, p.H, p.T, p.packed ? 1 : p.B, r.V, (long long)p.H * r.V,
                                (long long)p.T * p.H * r.V, kBlk);
    return e;
}

template <int KP, int VP, bool kOut, int kPieces>
cudaError_t launch(const TcParams& p, cudaStream_t st) {
    auto kernel = scan_tc_kernel<KP, VP, kOut, kPieces>;
    constexpr size_t smem = Layout<KP, VP, kPieces>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)p.s.plan.items, kThreads, smem, st>>>(p);
    return cudaGetLastError();
}

template <int KP, int VP>
cudaError_t launch_dims(const TcParams& p, bool state_only, cudaStream_t st) {
    bool state = false;  // whether a state is a result
    for (int r = 0; r < p.s.plan.nroles; ++r) state = state || p.s.role[r].fin;
    if (state_only) return state ? launch<KP, VP, false, 3>(p, st) : launch<KP, VP, false, 2>(p, st);
    return state ? launch<KP, VP, true, 3>(p, st) : launch<KP, VP, true, 2>(p, st);
}

}  // namespace

bool scan_tc_supported(const ScanRole& r, const ScanPlan& p, bool bf16) {
    if (!bf16 || r.K > 128 || r.V > 128 || r.K % 8 != 0 || r.V % 8 != 0) return false;
    CUtensorMap m[4];
    return role_maps(r, p, m) == cudaSuccess;
}

cudaError_t launch_scan_tc(const ScanLaunch& s, bool state_only, cudaStream_t st) {
    if (s.plan.items > 0x7fffffffLL) return cudaErrorInvalidValue;
    TcParams p;
    p.s = s;
    for (int r = 0; r < kScanRoles; ++r) {
        cudaError_t e = role_maps(s.role[r < s.plan.nroles ? r : 0], s.plan, p.map[r]);
        if (e != cudaSuccess) return e;
    }
    const int k = padded(s.role[0].K), v = padded(s.role[0].V);
    if (k == 64) return v == 64 ? launch_dims<64, 64>(p, state_only, st) : launch_dims<64, 128>(p, state_only, st);
    return v == 64 ? launch_dims<128, 64>(p, state_only, st) : launch_dims<128, 128>(p, state_only, st);
}

}  // namespace ssd

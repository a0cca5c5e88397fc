// linear_tc.cu -- the linear-attention scan on the fifth-generation tensor
// cores (bf16, K and V up to 128, padded with zeros to 64 or 128).
//
// One block per item (a chain or a piece of one), chunks of 128 tokens in scan
// order.  With positions i, j in a chunk of n tokens, l = exp(decay) and H the
// fp32 state entering it:
//     S   = Q K^T                                   scores
//     P   = S o L,  L_ij = out_scale l^|i-j| on the causal side, else 0   (bf16, in TMEM)
//     out = P V + out_scale diag(l^(i+1)) Q H       two accumulators, joined in fp32
//     Z   = (w o K)^T V,  w_j = l^(n-1-j)           the chunk's own state
//     H  <- l^n H + Z                               in registers, fp32
// and the mirror image for a scan backwards.  No power of l has a negative
// exponent; a table of them is made in 64 bits.
//
// Precision.  P, and H as an operand, are rounded to bf16 (their errors are
// those of the result's own rounding).  The state itself is fp32 and outlives
// the call, so w o K must not lose bits: it (or w o V, whichever is 64 wide)
// enters the product as kPieces bf16 numbers, the first ones its leading bits,
// the last one rounded: 3 hold the fp32 product whole and are used where the
// state is a result, 2 (error up to 2^-16) where it only enters outputs.
// l^n multiplies H at every chunk and is kept as a sum of two fp32 numbers, or
// its rounding would grow with the number of chunks.
//
// Warp roles (640 threads):
//   0-3    scores -> P (thread = row i), and with V = 128 the last quarter of
//   4-7    w o K or w o V in pieces: groups of 32 tokens, four warps to each; rows
//          behind a partial chunk's end become zeros in K and V (with packed
//          sequences they hold the next one's tokens)
//   8-15   state and output, two warps to a TMEM lane quadrant
//   16     lane 0 loads tiles by TMA; lane 1 stores output tiles (plain stores of rows
//          by their threads touch 32 lines each and kept the load/store unit busy
//          for 2000 cycles a chunk)
//   17     TMEM; issues Q H and P V
//   18     issues S, a chunk ahead where V = 64 leaves TMEM for a second score buffer
//   19     issues Z.  An MMA of 128 rows and 16 tokens takes 48 cycles at N = 64 and 64
//          at N = 128 (measured): a chunk's products are 2700 cycles at K = 128, V =
//          64 and 3100 at 128, 128; its loads and stores at the card's copy rate
//          are 4100 and 5500.
//
// With V = 128 the lanes of Z are the state's columns (v), else its rows (k): an
// MMA takes 128 rows, and the other order would waste half of them.
//
// Measured (4 x 8192 tokens, 37 heads: a chain per SM; with the final state, without
// it, and in brackets what the bytes take at the copy rate): 128 x 64 178, 164 us (142),
// 64 x 64 153, 139 (95), 64 x 128 190, 181 (142), 128 x 128 302, 283 (190).  What
// bounds it is the chain of dependent products of a chunk; no unit is busy for more
// than half of the time.
#include <climits>

#include "../common.cuh"
#include "../debug_checks.cuh"
#include "../linear.h"
#include "../tc_common.cuh"
#include "../tmap.h"

namespace ssd {
namespace {

constexpr int kBlk = kScanChunk;         // 128 tokens: the MMA's M
constexpr int kThreads = 640;
constexpr int kState = 8, kStateWarps = 8;  // first warp of the state's, how many
constexpr int kLoads = 16, kOutputs = 17, kScores = 18, kStates = 19;
constexpr uint32_t kPanel = kBlk * 128;  // 128 rows of 64 bf16
constexpr int kPartT = 16;               // tokens of a part: the MMA's K
constexpr uint32_t kPartPanel = kPartT * 128;
constexpr int kGroups = kBlk / (2 * kPartT);  // a chunk's groups of two parts

constexpr int kMaxBufs = 10;
struct __align__(8) Bars {
    uint64_t full[kMaxBufs], empty[kMaxBufs];
    // s_full alternates even with one score buffer: the next chunk's S may be done
    // before the warps that make the pieces have seen this one's
    uint64_t s_full[2], s_free[2], p_full[2], o_full, o_free;
    // by group of the chunk, not by buffer: a warp then waits for every phase of a
    // barrier that it waits on
    uint64_t x_full[kGroups], x_free[kGroups], clean;
    uint64_t z_full[2], z_free[2], h_full, h_free, staged, stored, landed;
    uint64_t done, z_done, s_done;
};

// Matrix descriptors (128-byte swizzle, 1024 bytes from one group of eight rows to
// the next) by their low words: start address and leading-dimension offset.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
    return ((saddr >> 4) & 0x3FFF) | (lbo_bytes >> 4) << 16;
}
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t adv_bytes) {
    constexpr uint32_t hi = (1024u >> 4) | 1u << 14 | 2u << 29;
    return (uint64_t)hi << 32 | (lo + (adv_bytes >> 4));
}

struct TcParams {
    CUtensorMap map[kScanRoles][4];
    ScanLaunch s;
};

// Shared and tensor memory of a variant.  K = V = 128: the first piece of w o K
// goes into K's own place once the scores are done; with outputs, a ring of
// kSlots tiles in the order q, k, v, q, ... (a whole second chunk does not fit), the
// output tile in V's place.  The others hold whole chunks, all pieces and an
// output tile; a scan for states alone holds k and v of whole chunks.
template <int KP, int VP, bool kOut, int kPieces>
struct Layout {
    static constexpr bool kInPlace = KP == 128 && VP == 128, kRing = kInPlace && kOut;
    static constexpr int kSlots = 5;
    static constexpr uint32_t kKB = KP / 64 * kPanel, kVB = VP / 64 * kPanel;
    static constexpr uint32_t kChunk = (kOut ? 2 : 1) * kKB + kVB;
    static constexpr int kStages = kRing ? 0 : kOut ? (KP == 64 && VP == 64 ? 3 : 2) : kInPlace ? 2 : KP + VP == 128 ? 5 : 3;
    static constexpr int kTiles = kOut ? 3 : 2;  // of a chunk
    static constexpr int kBufs = kRing ? kSlots : kTiles * kStages;
    static_assert(kBufs <= kMaxBufs, "barriers");
    // the scaled operand and its parts: pieces kFirst .. kPieces - 1 in buffers
    static constexpr bool kScaleV = VP == 64;
    static constexpr int kXW = kInPlace ? 128 : 64;
    static constexpr int kFirst = kInPlace ? 1 : 0;
    static constexpr uint32_t kPieceB = kXW / 64 * kPartPanel;
    static constexpr uint32_t kPartB = (kPieces - kFirst) * kPieceB;
    static constexpr int kGroupBufs = !kOut ? 4 : kRing ? 2 : KP == 128 ? 2 : 4;
    static constexpr uint32_t OFF_PART = kRing ? kSlots * 2 * kPanel : kStages * kChunk;
    static constexpr uint32_t OFF_H = OFF_PART + 2 * kGroupBufs * kPartB;
    static constexpr uint32_t OFF_OUT = OFF_H + (kOut ? (uint32_t)KP * VP * 2 : 0);
    static constexpr uint32_t OFF_TAB = OFF_OUT + (kRing || !kOut ? 0 : kVB);
    static constexpr uint32_t OFF_NEAR = OFF_TAB + 132 * 4;
    static constexpr uint32_t OFF_DEC = OFF_NEAR + 160 * 4;
    static constexpr uint32_t OFF_BAR = OFF_DEC + 4 * 8;
    static constexpr uint32_t OFF_MISC = OFF_BAR + (sizeof(Bars) + 15) / 16 * 16;
    static constexpr uint32_t OFF_ITEM = OFF_MISC + 16;
    static constexpr size_t kBytes = 1024 + OFF_ITEM + sizeof(ScanItem);
    static_assert(kBytes <= 232448, "shared memory above the 227 KB per-block limit");
    static_assert(OFF_PART % 1024 == 0 && OFF_H % 1024 == 0 && OFF_OUT % 1024 == 0, "swizzled tiles start on 1024 bytes");

    // TMEM columns: scores (P in their first 64), P V, Q H, Z.  (Tried with V = 64:
    // P beside one score buffer and all pieces' products side by side, which reads
    // 64 KB less of shared memory a chunk: 5 % slower at K = 128, 20 % at K = 64,
    // since the scores no longer run a chunk ahead.)
    static constexpr int kS = VP == 64 ? 2 : 1;
    static constexpr int kZ = VP == 64 ? 2 : 1;
    // K = 64, V = 128 has columns for two pieces side by side: one MMA reads the whole
    // operand for both, the third piece is added to the second's columns
    static constexpr int kSide = KP == 64 && VP == 128 ? 2 : 1;
    static constexpr uint32_t COL_S = 0, COL_O1 = 128 * kS, COL_O2 = COL_O1 + VP, COL_Z = 384;

    // buffer, its use count and its place, of tile `which` (0 q, 1 k, 2 v) of chunk c;
    // a state-only scan loads no q
    struct Buf { uint32_t i, use, off; };
    static __device__ __forceinline__ Buf buf(uint32_t c, uint32_t which) {
        Buf b;
        if constexpr (kRing) {
            const uint32_t n = 3 * c + which;
            b.use = n / kSlots;
            b.i = n - kSlots * b.use;
            b.off = b.i * 2 * kPanel;
        } else {
            b.use = c / (uint32_t)kStages;
            const uint32_t st = c - b.use * kStages, k = which - (3 - kTiles);  // k-th tile of its chunk
            b.i = kTiles * st + k;
            b.off = st * kChunk + (k > 0 ? kKB : 0) + (k > 1 ? kKB : 0);
        }
        return b;
    }
};

// A bounded wait in few instructions (each role's loop is executed once per chunk,
// and all of them together have to stay in the instruction cache; a call would
// spill the state that the warps hold in registers).  A try sleeps up to a
// microsecond; a wait is for other warps of the block and its own copies, some tens of
// tries at most, and after 2^20 (25 ms at the very least, a second as a rule) it has
// failed.  What takes as long as it takes, the call's earlier kernels, the whole block
// has waited for before its first such wait.
__device__ __forceinline__ bool wait_here(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 1048576;\n"
        "WAIT_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "@p bra DONE_%=;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra WAIT_%=;\n"
        "DONE_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// A masked place of P is a zero, but its product with an infinity or NaN of v is a
// NaN, which no earlier token's output may see.  Where P V is not finite in
// some of a warp's 32 rows of a column, the rows are stored without it and the column's
// `first` keeps the chunk; at the end of the item this adds the causal side's
// products to them, on CUDA cores (some 100 us; rare).  A later chunk's such rows of
// the column need none of it: from there on the state's column is not finite, and so
// is every output.  A warp mends its own rows (lane's: lr) and 32 columns from col,
// lane l holding column l's chunk.
// Looking for such rows costs 1.5 % at 128 x 64, 8 % at 64 x 128, nothing measurable
// at 128 x 128; a vote for every 16 columns instead of one a chunk cost 11 % at
// 64 x 128, mending at once, which makes registers spill, 25 %.
__device__ __forceinline__ void mend_rows(const ScanLaunch& s, const ScanItem& it, int nch, int lr, int first,
                                          const float* table, int col) {
    const ScanRole& R = s.role[it.role];
    const bool rev = R.reverse != 0;
    while (true) {
        const int c = (int)__reduce_min_sync(0xffffffffu, (unsigned)first);
        if (c == INT_MAX) break;
        const uint32_t mine = __ballot_sync(0xffffffffu, first == c);  // the columns whose chunk it is
        if (first == c) first = INT_MAX;
        const int t = it.t0 + (rev ? nch - 1 - c : c) * kBlk, n = min(kBlk, it.t1 - t);
        const long long row0 = it.row0 + t;
        const float* near = table + (rev ? 32 : kBlk - 1) - lr;
        for (int x = 0; lr < n && x < 32; x += 16) {
            const uint32_t m = (mine >> x) & 0xffffu;
            if (m == 0) continue;
            const __nv_bfloat16* q = (const __nv_bfloat16*)R.q.p + it.batch * R.q.batch + (row0 + lr) * R.q.token +
                                     it.head / R.q.share * R.q.head;
            const __nv_bfloat16* k = (const __nv_bfloat16*)R.k.p + it.batch * R.k.batch + row0 * R.k.token +
                                     it.head / R.k.share * R.k.head;
            const __nv_bfloat16* v = (const __nv_bfloat16*)R.v.p + it.batch * R.v.batch + row0 * R.v.token +
                                     it.head / R.v.share * R.v.head + col + x;
            float a[16] = {};
#pragma unroll 1
            for (int j = rev ? lr : 0; j < (rev ? n : lr + 1); ++j) {
                float sc = 0.f;
#pragma unroll 1
                for (int e = 0; e < R.K; ++e) sc = fmaf(to_f32(q[e]), to_f32(k[j * R.k.token + e]), sc);
                const float p = to_f32(from_f32<__nv_bfloat16>(sc * near[j]));
                bool done = true;  // nothing finite is left where all are NaN
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if ((m >> e) & 1 && col + x + e < R.V) {
                        a[e] = fmaf(p, to_f32(v[j * R.v.token + e]), a[e]);
                        done = done && a[e] != a[e];
                    }
                if (done) break;
            }
            const long long at = (((long long)it.batch * s.plan.T + row0 + lr) * s.plan.H + it.head) * R.V + col + x;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (!((m >> e) & 1) || col + x + e >= R.V ||
                    !SSD_INB(at + e, (s.plan.packed ? 1LL : s.plan.B) * s.plan.T * s.plan.H * R.V))
                    continue;
                if (R.out_f32) {
                    float* y = (float*)R.out + at + e;
                    *y = __ldcg(y) + a[e];
                } else {
                    __nv_bfloat16* y = (__nv_bfloat16*)R.out + at + e;
                    *y = from_f32<__nv_bfloat16>(to_f32(__ldcg(y)) + a[e]);  // (not an L1 line of before)
                }
            }
        }
        __syncwarp();
    }
}

template <int KP, int VP, bool kOut, int kPieces>
__global__ void __launch_bounds__(kThreads, 1) scan_tc_kernel(const __grid_constant__ TcParams p) {
    using L = Layout<KP, VP, kOut, kPieces>;
    constexpr bool kLaneV = VP == 128;         // lanes of Z: v, else k
    constexpr int CH = kLaneV ? KP / 2 : 32;   // state columns of a thread
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sH = sm + L::OFF_H;
    float* sTab = reinterpret_cast<float*>(sm + L::OFF_TAB);  // l^0 .. l^128
    // out_scale l^d for the scores (0 for d < 0): d = 127 .. -32, or -32 .. 127 backwards
    float* sNear = reinterpret_cast<float*>(sm + L::OFF_NEAR);
    // what H is multiplied by in a whole chunk, in the first and in the last one
    float2* sDec = reinterpret_cast<float2*>(sm + L::OFF_DEC);
    Bars* bars = reinterpret_cast<Bars*>(sm + L::OFF_BAR);
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + L::OFF_MISC);
    volatile uint32_t* sMend = sTmem + 1;  // whether rows are to be mended
    ScanItem* sItem = reinterpret_cast<ScanItem*>(sm + L::OFF_ITEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    next_may_start();
    if (p.s.reset && blockIdx.x == 0 && threadIdx.x == 0) *p.s.status = kDevOk;
    if (warp == 0) {
        ScanItem f = scan_item(p.s.plan, blockIdx.x);
        if (f.valid) scan_item_tokens(f, p.s.plan.seg_tokens, p.s.role[f.role].reverse);
        if (lane == 0) *sItem = f;
    }
    __syncthreads();
    const ScanItem it = *sItem;
    if (!it.valid || (!kOut && it.seg == it.nseg - 1)) {
        if (blockIdx.x == 0) wait_for_earlier();
        return;
    }
    const ScanRole& R = p.s.role[it.role];
    const int K = R.K, V = R.V;
    const bool rev = R.reverse != 0;
    const float out_scale = R.out_scale;
    const bool out_f32 = R.out_f32 != 0, packed = p.s.plan.packed != 0;
    const float la = p.s.decay[it.head];
    const int H = p.s.plan.H;
    const long long chain = (long long)it.seq * H + it.head;
    const long long chains = (long long)p.s.plan.B * H;
    (void)chains;
    const int span = it.t1 - it.t0;
    const int nch = (span + kBlk - 1) / kBlk;

    // first token (in the sequence) and tokens of the c-th chunk in scan order
    auto chunk_at = [&](int c) -> int { return it.t0 + (rev ? nch - 1 - c : c) * kBlk; };
    auto chunk_n = [&](int t) -> int { return min(kBlk, it.t1 - t); };
    auto load_tile = [&](int c, int w, int head) {
        const auto b = L::buf(c, w);
        const int panels = (w == 2 ? VP : KP) / 64;
        tc::mbar_arrive_expect_tx(&bars->full[b.i], panels * kPanel);
        for (int x = 0; x < panels; ++x)
            tc::tma_load_4d(sm + b.off + x * kPanel, &p.map[it.role][w], &bars->full[b.i], 64 * x, head,
                            (int)(it.row0 + chunk_at(c)), it.batch);
    };
    if (warp == kLoads && lane == 0) {
        for (int i = 0; i < L::kBufs; ++i) {
            // a tile's place is free again when both its products are done (q: S, Q H;
            // k: S, Z; v: P V, Z) and, in the ring, v's output has left
            tc::mbar_init(&bars->full[i], 1);
            tc::mbar_init(&bars->empty[i], !kOut ? 1 : L::kRing ? 3 : 2);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars->s_full[i], 1);
            tc::mbar_init(&bars->s_free[i], 1);
            tc::mbar_init(&bars->p_full[i], 4);
        }
        tc::mbar_init(&bars->o_full, 1);
        tc::mbar_init(&bars->o_free, kStateWarps);
        for (int i = 0; i < kGroups; ++i) {
            tc::mbar_init(&bars->x_full[i], 4);
            tc::mbar_init(&bars->x_free[i], 1);
        }
        tc::mbar_init(&bars->clean, 8);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars->z_full[i], 1);
            tc::mbar_init(&bars->z_free[i], kStateWarps);
        }
        tc::mbar_init(&bars->h_full, kStateWarps);
        tc::mbar_init(&bars->h_free, 1);
        tc::mbar_init(&bars->staged, kStateWarps);
        tc::mbar_init(&bars->stored, 1);
        tc::mbar_init(&bars->landed, 1);
        *sMend = 0;
        tc::mbar_init(&bars->z_done, 1);
        tc::mbar_init(&bars->s_done, 1);
        tc::mbar_init(&bars->done, 1);
        tc::fence_mbar_init();
        tc::fence_proxy_async_smem();
        // the first chunk's tiles, while the others make the tables
        if (nch > 0)
            for (int w = kOut ? 0 : 1; w < 3; ++w)
                load_tile(0, w, it.head / (w == 0 ? R.q.share : w == 1 ? R.k.share : R.v.share));
    }
    __syncwarp();
    if (warp == kOutputs) {
        tc::tmem_alloc(sTmem, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x >= 64 && threadIdx.x - 64 <= kBlk + 32) {
        const int d = (int)threadIdx.x - 96;
        const float e = d < 0 ? 0.f : decay_power(la, d).x;
        if (d >= 0) sTab[d] = e;
        if (d < kBlk) sNear[rev ? d + 32 : kBlk - 1 - d] = e * out_scale;
    }
    // a backward scan's initial state meets its first token undecayed
    const int off0 = it.seg == 0 && rev ? 0 : 1;
    if (threadIdx.x >= 256 && threadIdx.x < 259) {
        const int i = threadIdx.x - 256;
        const int at_end = (span - 1) % kBlk + 1;  // tokens of the sequence's partial chunk, or 128
        const int n = nch == 0 || i == 0 ? kBlk : i == 1 ? (rev || nch == 1 ? at_end : kBlk) : (rev && nch > 1 ? kBlk : at_end);
        sDec[i] = decay_power(la, i == 1 || (i == 2 && nch == 1) ? n - 1 + off0 : n);
    }
    // an item that starts from a slot starts when the combination is done, however long
    // that takes: before any role's first wait, whose limits are for the block's own work
    if (kOut && it.slot_prev >= 0) wait_for_earlier();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *sTmem;
    // 64 state columns in a thread do not fit beside the rest in the 96 registers
    // that 19 warps leave each: those warps take 24 from the scores' and pieces'
    auto give = [] { if constexpr (CH == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); };
    auto take = [] { if constexpr (CH == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 120;"); };

    auto fail = [&]() { atomicExch(p.s.status, kDevTimeout); };
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return wait_here(bar, parity); };
    // the same decision in every lane: what follows is executed by whole warps
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_here(bar, parity));
    };
    // Arrivals on a tile's empty barrier once the products that this thread issued so
    // far are done.  Buffers of the ring hold q, k and v in turn and expect three
    // arrivals each time: S makes one of q's and k's, Q H and Z the other two, P V, Z
    // and the output's store one each of v's.
    auto release = [&](uint32_t e, uint32_t buf, int in_ring) {
        tc::mma_commit_if(e, &bars->empty[buf]);
        if (kOut && L::kRing && in_ring == 2) tc::mma_commit_if(e, &bars->empty[buf]);
    };
    // a chunk of n tokens whose output leaves by plain stores: fp32, or a packed
    // sequence's end, behind which the rows are another's
    auto direct = [&](int n) -> bool { return out_f32 || (packed && n < kBlk); };

    if (warp == kLoads) {
        if (lane == 0) {
            // ------------------------------------------------- TMA loads ----
            // (unrolled: with rolled loops the loads went out later, 40 us of 450)
            bool ok = true;
            const int hq = it.head / R.q.share, hk = it.head / R.k.share, hv = it.head / R.v.share;
            int c = 1;
#pragma unroll 1
            for (; ok && c < nch; ++c) {
#pragma unroll
                for (int w = kOut ? 0 : 1; w < 3; ++w) {
                    const auto b = L::buf(c, w);
                    if (b.use > 0 && !wait(&bars->empty[b.i], (b.use - 1) & 1)) { ok = false; break; }
                    load_tile(c, w, w == 0 ? hq : w == 1 ? hk : hv);
                }
            }
            if (!ok) {
                fail();
                // no copy may still be landing in shared memory when the block exits
                for (int cc = c > 4 ? c - 4 : 0; cc < c; ++cc)
                    for (int w = kOut ? 0 : 1; w < 3; ++w) {
                        const auto b = L::buf(cc, w);
                        tc::mbar_wait(&bars->full[b.i], b.use & 1, nullptr, 200000000ull);
                    }
            }
        } else if (kOut && lane == 1) {
            // ---------------------------------------------------- TMA stores ----
            bool ok = true;
            for (int c = 0; c < nch; ++c) {
                const int t = chunk_at(c);
                const auto bv = L::buf(c, 2);
                ok = wait(&bars->staged, c & 1);
                if (!ok) break;
                if (!direct(chunk_n(t))) {
                    const uint8_t* tile = sm + (L::kRing ? bv.off : L::OFF_OUT);
                    for (int x = 0; x < VP / 64; ++x)
                        if (64 * x < V)
                            tc::tma_store_4d(&p.map[it.role][3], tile + x * kPanel, 64 * x, it.head, (int)(it.row0 + t),
                                             it.batch);
                    tc::bulk_commit();
                    tc::bulk_wait_read<0>();
                }
                if (L::kRing) tc::mbar_arrive(&bars->empty[bv.i]);
                tc::mbar_arrive(&bars->stored);
            }
            if (ok && *sMend) {
                tc::bulk_wait<0>();
                tc::mbar_arrive(&bars->landed);
            }
            if (!ok) fail();
        }
    } else if (warp >= kOutputs) {
        // ------------------------------------------------------ MMA issue ----
        constexpr uint32_t id_s = tc::idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint32_t id_pv = tc::idesc_bf16_f32(128, VP, 0, 1);
        constexpr uint32_t id_qh = tc::idesc_bf16_f32(128, VP, 0, kLaneV ? 0 : 1);
        constexpr uint32_t id_z = tc::idesc_bf16_f32(128, L::kSide * L::kXW, 1, 1);
        constexpr uint32_t id_z1 = tc::idesc_bf16_f32(128, L::kXW, 1, 1);
        const uint32_t base = __shfl_sync(0xffffffffu, tc::smem_u32(sm), 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const int chunks = __shfl_sync(0xffffffffu, nch, 0);
        const uint32_t kmaj = desc_lo(base, 16);       // rows contiguous along the contraction
        const uint32_t mnmaj = desc_lo(base, kPanel);  // contraction along the rows
        const uint32_t lead = tc::elect_one();
        bool ok = true;
        if (warp == kScores) {
#pragma unroll 1
            for (int c = 0; kOut && c < chunks; ++c) {
                const auto bq = L::buf(c, 0), bk = L::buf(c, 1);
                // the scores overwrite the P that P V of the chunk kS before read
                ok = wait_warp(&bars->full[bq.i], bq.use & 1) && wait_warp(&bars->full[bk.i], bk.use & 1) &&
                     (c < L::kS || wait_warp(&bars->s_free[c % L::kS], (c / L::kS - 1) & 1));
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t dq = kmaj + (bq.off >> 4), dk = kmaj + (bk.off >> 4);
                const uint32_t d = tm + L::COL_S + (c % L::kS) * 128;
#pragma unroll 4
                for (int kk = 0; kk < KP / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kPanel + (kk & 3) * 32;
                    tc::mma_ss_if(lead, d, desc(dq, off), desc(dk, off), id_s, kk > 0);
                }
                tc::mma_commit_if(lead, &bars->s_full[c & 1]);
                release(lead, bq.i, 1);
                release(lead, bk.i, 1);
            }
        } else if (warp == kOutputs) {
#pragma unroll 1
            for (int c = 0; kOut && c < chunks; ++c) {
                const auto bq = L::buf(c, 0), bv = L::buf(c, 2);
                // Q H
                ok = wait_warp(&bars->full[bq.i], bq.use & 1) && wait_warp(&bars->h_full, c & 1) &&
                     (c == 0 || wait_warp(&bars->o_free, (c - 1) & 1));
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t dq = kmaj + (bq.off >> 4);
#pragma unroll 4
                for (int kk = 0; kk < KP / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kPanel + (kk & 3) * 32;
                    const uint64_t dh = kLaneV ? desc(kmaj, L::OFF_H + off) : desc(mnmaj, L::OFF_H + kk * 2048);
                    tc::mma_ss_if(lead, tm + L::COL_O2, desc(dq, off), dh, id_qh, kk > 0);
                }
                tc::mma_commit_if(lead, &bars->h_free);
                release(lead, bq.i, 2);
                // P V
                ok = wait_warp(&bars->full[bv.i], bv.use & 1) &&
                     wait_warp(&bars->p_full[c % L::kS], (c / L::kS) & 1) &&
                     (chunk_n(chunk_at(c)) == kBlk || wait_warp(&bars->clean, 0));
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t dv = mnmaj + (bv.off >> 4);
                const uint32_t a = tm + L::COL_S + (c % L::kS) * 128;
#pragma unroll 4
                for (int kk = 0; kk < kBlk / 16; ++kk)
                    tc::mma_ts_if(lead, tm + L::COL_O1, a + kk * 8, desc(dv, kk * 2048), id_pv, kk > 0);
                tc::mma_commit_if(lead, &bars->o_full);
                tc::mma_commit_if(lead, &bars->s_free[c % L::kS]);
                release(lead, bv.i, 1);
            }
        } else {
            const uint32_t partmn = desc_lo(base + L::OFF_PART, kPartPanel);
#pragma unroll 1
            for (int c = 0; ok && c < chunks; ++c) {
                const auto bk = L::buf(c, 1), bv = L::buf(c, 2);
                ok = wait_warp(&bars->full[bk.i], bk.use & 1) && wait_warp(&bars->full[bv.i], bv.use & 1) &&
                     (c < L::kZ || wait_warp(&bars->z_free[c % L::kZ], (c / L::kZ - 1) & 1)) &&
                     (chunk_n(chunk_at(c)) == kBlk || wait_warp(&bars->clean, 0));
                if (!ok) break;
                tc::tc_fence_after();
                // the operand that stays whole fills the MMA's rows
                const uint32_t whole = mnmaj + ((L::kScaleV ? bk.off : bv.off) >> 4);
                const uint32_t inplace = mnmaj + (bk.off >> 4);
                const uint32_t z = tm + L::COL_Z + (c % L::kZ) * 64;
#pragma unroll 1
                for (int u = 0; u < kGroups; ++u) {
                    const uint32_t s = u % L::kGroupBufs;
                    ok = wait_warp(&bars->x_full[u], c & 1);
                    if (!ok) break;
                    const uint32_t da = whole + ((u * 2 * kPartPanel) >> 4);
                    const uint32_t di = inplace + ((u * 2 * kPartPanel) >> 4);
                    const uint32_t dx = partmn + ((s * 2 * L::kPartB) >> 4);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int x = 0; x < kPieces; x += x == 0 ? L::kSide : 1)
                            tc::mma_ss_if(lead, x == 0 ? z : z + (L::kSide - 1) * L::kXW, desc(da, i * kPartPanel),
                                          x < L::kFirst ? desc(di, i * kPartPanel)
                                                        : desc(dx, i * L::kPartB + (x - L::kFirst) * L::kPieceB),
                                          x == 0 ? id_z : id_z1, (u > 0 || i > 0 || x > 0) ? 1u : 0u);
                    tc::mma_commit_if(lead, &bars->x_free[u]);
                }
                if (!ok) break;
                tc::mma_commit_if(lead, &bars->z_full[c % L::kZ]);
                release(lead, bk.i, 2);
                release(lead, bv.i, 1);
            }
        }
        if (!ok) fail();
        // every product issued must be complete before TMEM is released
        uint64_t* done = warp == kOutputs ? &bars->done : warp == kScores ? &bars->s_done : &bars->z_done;
        tc::mma_commit_if(lead, done);
        tc::mbar_wait(done, 0, nullptr, 200000000ull);
    } else if (warp < 8) {
        // ------------------------------------------------- P, thread = row ----
        // --------------------------------- and w o K or w o V in pieces ----
        give();
        const uint32_t ts = tmem + ((uint32_t)(warp * 32) << 16) + L::COL_S;
        // out_scale l^|i-j| of row i against the columns of block jb: 32 consecutive
        // entries of a table, neighbouring lanes one apart
        const float* near = sNear + (rev ? 32 : kBlk - 1) - (32 * warp + lane);
        const uint32_t diag = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
        // four warps to a group: its part, the row of it, the first 16-byte column
        const int part = (warp >> 1) & 1, r = (lane & 7) + 8 * (warp & 1), ch = lane >> 3;
        bool ok = true;
#pragma unroll 1
        for (int c = 0; ok && c < nch; ++c) {
            const int n = chunk_n(chunk_at(c));
            const auto bk = L::buf(c, 1), bv = L::buf(c, 2);
            const auto bx = L::kScaleV ? bv : bk;
            if (n < kBlk) {
                // k's rows behind the end: the scores' columns there are masked,
                // whatever they are
                ok = wait_warp(&bars->full[bk.i], bk.use & 1) && wait_warp(&bars->full[bv.i], bv.use & 1) &&
                     (!kOut || wait_warp(&bars->s_full[c & 1], (c >> 1) & 1));
                if (!ok) break;
                // a row's panels of k, then of v: eight lanes each; where pieces go in place,
                // k's rows belong to their part's warps
                const int x = lane >> 3;
                if (x < (KP + VP) / 64 && !(L::kInPlace && x < KP / 64)) {
                    uint8_t* at = sm + (x < KP / 64 ? bk.off + x * kPanel : bv.off + (x - KP / 64) * kPanel) + (lane & 7) * 16;
                    for (int f = n + warp; f < kBlk; f += 8)
                        *reinterpret_cast<uint4*>(at + f * 128) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars->clean);
            }
            if (kOut && warp < 4) {
                const uint32_t tc0 = ts + (c % L::kS) * 128;
                ok = wait_warp(&bars->s_full[c & 1], (c >> 1) & 1);
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
                        tc::tmem_ld32(tc0 + 32 * jb, s);
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
                    tc::tmem_st16(tc0 + 16 * jb, r);
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars->p_full[c % L::kS]);
            }
            ok = wait_warp(&bars->full[bx.i], bx.use & 1) &&
                 // in the ring the first piece takes k's place: the scores have read it
                 (!(kOut && L::kRing) || wait_warp(&bars->s_full[c & 1], (c >> 1) & 1));
            if (!ok) break;
            // warps 0-3 make P and, with V = 128, the last group, 4-7 the others;
            // without P every other group each
            constexpr int kMine = VP == 64 ? kGroups : kGroups - 1;
            const int u0 = kOut ? (warp < 4 ? kMine : 0) : (warp < 4 ? 1 : 0), u1 = kOut && warp >= 4 ? kMine : kGroups;
#pragma unroll 1
            for (int u = u0; u < u1; u += kOut ? 1 : 2) {
                const uint32_t s = u % L::kGroupBufs;
                // the buffer's last group: of this chunk, or of the one before
                const int before = (u + kGroups - L::kGroupBufs) % kGroups, cb = before < u ? c : c - 1;
                if (cb >= 0) {
                    ok = wait_warp(&bars->x_free[before], cb & 1);
                    if (!ok) break;
                }
                const int row = kPartT * (2 * u + part) + r;
                const bool inside = row < n;
                const float w = inside ? sTab[rev ? row : n - 1 - row] : 0.f;
                const float2 w2 = make_float2(w, w), minus = make_float2(-1.f, -1.f);
                uint8_t* src = sm + bx.off + row * 128;
                uint8_t* out = sm + L::OFF_PART + (2 * s + part) * L::kPartB + r * 128;
                uint4 v[L::kXW / 32];  // all loads before the first store (which may be to the same place)
#pragma unroll
                for (int i = 0; i < L::kXW / 32; ++i)  // eight neighbouring rows take eight different 16-byte columns
                    v[i] = *reinterpret_cast<const uint4*>(src + (i >> 1) * kPanel + ((4 * (i & 1) + ch) ^ (r & 7)) * 16);
#pragma unroll
                for (int i = 0; i < L::kXW / 32; ++i) {
                    const int x = i >> 1, cc = ((4 * (i & 1) + ch) ^ (r & 7)) * 16;
                    if (!inside) v[i] = make_uint4(0, 0, 0, 0);
                    const uint32_t in4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t q[kPieces][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 f = tc::mul2(tc::unpack_bf16x2(in4[e]), w2);
#pragma unroll
                        for (int y = 0; y + 1 < kPieces; ++y) {
                            // the leading 8 bits of each, and what they leave (exactly)
                            q[y][e] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
                            f = tc::fma2(make_float2(__uint_as_float(__float_as_uint(f.x) & 0xffff0000u),
                                                     __uint_as_float(__float_as_uint(f.y) & 0xffff0000u)), minus, f);
                        }
                        q[kPieces - 1][e] = tc::pack_bf16x2(f.x, f.y);
                    }
#pragma unroll
                    for (int y = 0; y < kPieces; ++y) {
                        uint8_t* to = y < L::kFirst ? src + x * kPanel : out + (y - L::kFirst) * L::kPieceB + x * kPartPanel;
                        *reinterpret_cast<uint4*>(to + cc) = make_uint4(q[y][0], q[y][1], q[y][2], q[y][3]);
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars->x_full[u]);
            }
        }
        if (!ok) fail();
    } else if (warp < kState + kStateWarps) {
        // ------------------------------------------------ state and output ----
        take();
        const int quad = warp & 3, half = (warp - 8) >> 2;
        const int lr = quad * 32 + lane;  // lane of TMEM
        const int c0 = half * CH;
        const bool holds = kLaneV || lr < KP;  // K = 64: lanes behind it hold nothing
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        float h[CH];
        const bool from_init = it.slot_prev < 0;
        // element of column c: (k, v)
        auto k_of = [&](int c) -> int { return kLaneV ? c0 + c : lr; };
        auto v_of = [&](int c) -> int { return kLaneV ? lr : c0 + c; };
#pragma unroll
        for (int c = 0; c < CH; ++c) h[c] = 0.f;
        if (kOut && holds && (it.seg > 0 || R.init)) {
            const float* src = from_init ? R.init + chain * K * V : p.s.states + it.slot_prev * K * V;
            const long long sk = from_init ? R.init_k : V, sv = from_init ? R.init_v : 1;
            const float mul = from_init ? R.init_scale : 1.f;
            src += k_of(0) * sk + v_of(0) * sv;
            const long long step = kLaneV ? sk : sv;
            const int have = kLaneV ? (lr < V ? K - c0 : 0) : (lr < K ? V - c0 : 0);
            if (step == 1) {  // the thread's columns are neighbours (K and V are multiples of 8)
#pragma unroll
                for (int c = 0; c < CH; c += 4)
                    if (c < have && SSD_INB(k_of(c) * sk + v_of(c) * sv + 3, (long long)K * V)) {
                        const float4 f = *reinterpret_cast<const float4*>(src + c);
                        h[c] = f.x * mul;
                        h[c + 1] = f.y * mul;
                        h[c + 2] = f.z * mul;
                        h[c + 3] = f.w * mul;
                    }
            } else {  // the lanes' are
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (c < have && SSD_INB(k_of(c) * sk + v_of(c) * sv, (long long)K * V)) h[c] = *src * mul;
                    src += step;
                }
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
        // the chunk whose rows of the warp's columns lane, lane + 32 are to be mended
        int first[VP / 64];
#pragma unroll
        for (int e = 0; e < VP / 64; ++e) first[e] = INT_MAX;
        if (kOut && nch > 0) put_h();
        int off = off0;
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            const int t = chunk_at(c), n = chunk_n(t);
            ok = wait_warp(&bars->z_full[c % L::kZ], (c / L::kZ) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            const float2 dec = sDec[c == 0 ? 1 : c + 1 == nch ? 2 : 0];
            const float2 dx = make_float2(dec.x, dec.x), dy = make_float2(dec.y, dec.y);
#pragma unroll
            for (int x = 0; x < CH / 16; ++x) {
                float z[L::kSide][16];
#pragma unroll
                for (int y = 0; y < L::kSide; ++y)
                    tc::tmem_ld16(tl + L::COL_Z + (c % L::kZ + y) * 64 + c0 + 16 * x, z[y]);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    float2 add = make_float2(z[0][e], z[0][e + 1]);
                    if constexpr (L::kSide == 2) {
                        add.x += z[1][e];
                        add.y += z[1][e + 1];
                    }
                    const float2 o = make_float2(h[16 * x + e], h[16 * x + e + 1]);
                    const float2 w = tc::fma2(o, dx, tc::fma2(o, dy, add));
                    h[16 * x + e] = w.x;
                    h[16 * x + e + 1] = w.y;
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars->z_free[c % L::kZ]);
            if (kOut) {
                if (c + 1 < nch) {
                    ok = wait_warp(&bars->h_free, c & 1);  // Q H has read this chunk's H
                    if (!ok) break;
                    put_h();
                }
                ok = wait_warp(&bars->o_full, c & 1);
                if (!ok) break;
                tc::tc_fence_after();
                const float e = lr < n ? sTab[(rev ? n - 1 - lr : lr) + off] * out_scale : 0.f;
                const long long row = (long long)it.batch * p.s.plan.T + it.row0 + t + lr;
                const long long at0 = (row * H + it.head) * V;
                const bool plain = direct(n);
                // the ring's tile takes the place of this chunk's V, consumed with z_full and
                // o_full; the others' is free once the last one has left (waited for in both:
                // no barrier may get two phases ahead of a warp that waits on it)
                uint8_t* tile = sm + (L::kRing ? L::buf(c, 2).off : L::OFF_OUT) + lr * 128;
                if (c > 0) {
                    ok = wait_warp(&bars->stored, (c - 1) & 1);
                    if (!ok) break;
                }
                auto finish = [&](int col, float (&a)[16], const float (&b)[16]) {
#pragma unroll
                    for (int q = 0; q < 16; q += 2) {
                        const float2 y = tc::fma2(make_float2(e, e), make_float2(b[q], b[q + 1]), make_float2(a[q], a[q + 1]));
                        a[q] = y.x;
                        a[q + 1] = y.y;
                    }
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
                                !SSD_INB(at0 + cy + 7, (packed ? 1LL : p.s.plan.B) * p.s.plan.T * H * V))
                                continue;
                            if (out_f32) {
                                float4* f = reinterpret_cast<float4*>((float*)R.out + at0 + cy);
                                f[0] = make_float4(a[8 * y], a[8 * y + 1], a[8 * y + 2], a[8 * y + 3]);
                                f[1] = make_float4(a[8 * y + 4], a[8 * y + 5], a[8 * y + 6], a[8 * y + 7]);
                            } else {
                                *reinterpret_cast<uint4*>((__nv_bfloat16*)R.out + at0 + cy) =
                                    make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                            }
                        }
                    }
                };
                float2 zero = make_float2(0.f, 0.f);  // stays so while P V is finite
#pragma unroll 1
                for (int x = 0; x < VP / 32; ++x) {
                    const int col = half * (VP / 2) + 16 * x;
                    float a[16], b[16];
                    tc::tmem_ld16(tl + L::COL_O1 + col, a);
                    tc::tmem_ld16(tl + L::COL_O2 + col, b);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 16; q += 2)
                        zero = tc::fma2(make_float2(a[q], a[q + 1]), make_float2(0.f, 0.f), zero);
                    finish(col, a, b);
                }
                if (__any_sync(0xffffffffu, lr < n && !(zero.x + zero.y == 0.f))) {  // again: see mend_rows
#pragma unroll 1
                    for (int x = 0; x < VP / 32; ++x) {
                        const int col = half * (VP / 2) + 16 * x;
                        float a[16], b[16];
                        tc::tmem_ld16(tl + L::COL_O1 + col, a);
                        tc::tmem_ld16(tl + L::COL_O2 + col, b);
                        tc::tmem_ld_wait();
                        const bool high = VP == 128 && x >= 2;
                        const uint32_t open =
                            __ballot_sync(0xffffffffu, (high ? first[VP / 64 - 1] : first[0]) == INT_MAX) >> (16 * (x & 1));
                        uint32_t now = 0;
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            // (not rows whose q is what is not finite: there Q H is not either)
                            if (__any_sync(0xffffffffu, lr < n && !(a[q] * 0.f == 0.f) && b[q] * 0.f == 0.f) &&
                                (open >> q) & 1) {
                                a[q] = 0.f;
                                now |= 1u << q;
                            }
                        if ((now >> (lane & 15)) & 1 && lane >> 4 == (x & 1)) {
                            if (high) first[VP / 64 - 1] = c;
                            else first[0] = c;
                            *sMend = 1;
                        }
                        finish(col, a, b);
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
        wait_for_earlier();
        float* dst = nullptr;
        float mul = 1.f;
        if (!kOut) {
            dst = p.s.states + it.slot * K * V;
        } else if (R.fin && it.seg == it.nseg - 1) {
            dst = R.fin + chain * K * V;
            mul = R.fin_scale * (rev && it.len > 0 ? sTab[1] : 1.f);
        }
        if (ok && dst && holds && SSD_INB(kOut ? chain : it.slot, kOut ? chains : p.s.plan.slots())) {
            dst += (long long)k_of(0) * V + v_of(0);
            const int have = kLaneV ? (lr < V ? K - c0 : 0) : (lr < K ? V - c0 : 0);
            if constexpr (kLaneV) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (c < have) *dst = h[c] * mul;
                    dst += V;
                }
            } else {  // (32 single stores of rows by their threads: 8000 cycles)
#pragma unroll
                for (int c = 0; c < CH; c += 4)
                    if (c < have)
                        *reinterpret_cast<float4*>(dst + c) =
                            make_float4(h[c] * mul, h[c + 1] * mul, h[c + 2] * mul, h[c + 3] * mul);
            }
        }
        if (kOut && ok && *sMend && wait_warp(&bars->landed, 0))
#pragma unroll
            for (int e = 0; e < VP / 64; ++e)
                mend_rows(p.s, it, nch, lr, first[e], sNear, half * (VP / 2) + 32 * e);
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kOutputs) {
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
    const long long grid = kOut ? p.s.plan.items : p.s.plan.state_items();
    auto kernel = scan_tc_kernel<KP, VP, kOut, kPieces>;
    constexpr size_t smem = Layout<KP, VP, kOut, kPieces>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_in_call(kernel, (unsigned)grid, kThreads, smem, st, !p.s.reset, p);
}

template <int KP, int VP>
cudaError_t launch_dims(const TcParams& p, bool state_only, cudaStream_t st) {
    bool state = false;  // whether a state is a result
    for (int r = 0; r < p.s.plan.nroles; ++r) state = state || p.s.role[r].fin;
    if (state_only) return state ? launch<KP, VP, false, 3>(p, st) : launch<KP, VP, false, 2>(p, st);
    return state ? launch<KP, VP, true, 3>(p, st) : launch<KP, VP, true, 2>(p, st);
}

}  // namespace

bool scan_tc_maps(const ScanLaunch& s, ScanMaps& m) {
    static_assert(sizeof(m.map) == sizeof(CUtensorMap) * kScanRoles * 4, "tensor maps");
    for (int i = 0; i < s.plan.nroles; ++i) {
        const ScanRole& r = s.role[i];
        if (!s.bf16 || r.K > 128 || r.V > 128 || r.K % 8 != 0 || r.V % 8 != 0) return false;
        if (role_maps(r, s.plan, reinterpret_cast<CUtensorMap*>(m.map[i])) != cudaSuccess) return false;
    }
    return true;
}

cudaError_t launch_scan_tc(const ScanLaunch& s, const ScanMaps& m, bool state_only, cudaStream_t st) {
    if (s.plan.items > 0x7fffffffLL) return cudaErrorInvalidValue;
    TcParams p;
    p.s = s;
    memcpy(p.map, m.map, sizeof(CUtensorMap) * 4 * s.plan.nroles);
    const int k = padded(s.role[0].K), v = padded(s.role[0].V);
    if (k == 64) return v == 64 ? launch_dims<64, 64>(p, state_only, st) : launch_dims<64, 128>(p, state_only, st);
    return v == 64 ? launch_dims<128, 64>(p, state_only, st) : launch_dims<128, 128>(p, state_only, st);
}

}  // namespace ssd

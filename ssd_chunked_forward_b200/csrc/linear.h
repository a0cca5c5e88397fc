// linear.h -- what the linear-attention kernels share: the scan's operands,
// how a launch is cut into items, and the launchers (internal; the public ABI
// is include/ssd.h).
//
// Everything here is one scan.  With l = exp(decay[h]) and a state h[K][V],
//     h_t = l h_{t-1} + k_t v_t^T,     out_t = out_scale * q_t^T h_t
// the forward is that scan of (q, k, v), and each gradient is the same scan
// with the roles of the tensors exchanged, backwards in time for dk and dv:
//     dq: (dy, v, k) forwards     dk: (v, dy, q) backwards     dv: (k, q, dy) backwards
// so one kernel serves them all, given a ScanRole for each.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#ifdef __CUDACC__
#define SSD_HD __host__ __device__
#else
#define SSD_HD
#endif

namespace ssd {

// one tensor of rows [batch][token][head][d], strides in elements (d is contiguous)
struct RowTensor {
    const void* p;
    long long batch, token, head;
    int share;  // head h of the scan reads head h / share of the tensor
};

struct ScanRole {
    RowTensor q, k, v;
    int K, V;          // contraction and value sizes of this scan's state
    int reverse;       // 1: from the last token to the first
    float out_scale;
    void* out;         // contiguous [rows][H][V], or null with a state-only scan
    int out_f32;       // out holds fp32 whatever the inputs' type
    // state of each chain before its first token, times init_scale; element
    // (k, v) of chain c at init[c * K * V + k * init_k + v * init_v]; null = zero.
    // A backward scan's initial state is added at the last token undecayed.
    const float* init;
    long long init_k, init_v;
    float init_scale;
    // state after the chain's last token times fin_scale (a backward scan: times
    // the decay of one further token), [chain][K][V]; null = not wanted
    float* fin;
    float fin_scale;
};

constexpr int kScanRoles = 3;
constexpr int kScanChunk = 128;  // tokens of a chunk on tensor cores
constexpr int kSimtChunk = 32;   // and on CUDA cores,
constexpr int kSimtColumns = 64; // state columns of a block there

// Shared memory of a block on CUDA cores: q and k rows, v, scores, state, powers.
struct SimtLayout {
    int K4, ldk;  // K rounded up to 4, row pitch of q and k
    size_t bytes;
};
SSD_HD inline SimtLayout simt_layout(int K) {
    SimtLayout l;
    l.K4 = (K + 3) & ~3;
    // an odd number of 16-byte units, so that eight rows' 16-byte reads meet no bank twice
    l.ldk = l.K4 + (l.K4 % 8 == 0 ? 4 : 8);
    l.bytes = (size_t)(2 * kSimtChunk * l.ldk + kSimtChunk * kSimtColumns + kSimtChunk * (kSimtChunk + 4) +
                       l.K4 * kSimtColumns + kSimtChunk + 4) * sizeof(float);
    return l;
}

// How the chains (sequence, head, role) are cut into items, one per block.
// Rows of equal length ([B][T]): the first `nfull` chains are one item each,
// the others `nseg` items of seg_tokens tokens.  Packed rows: every sequence
// is cut every seg_tokens tokens, and the items are found on the device.
// A chain of several items first has the state of each item but its last
// built from zero (state-only items), then those states combined into the
// state entering each item.
//
// Packed rows have their numbers from the offsets alone, so that a block finds its
// item by a search in them and nothing has to be counted first.  With d = seg_tokens
// and f(x) = floor(x / d), sequence s (rows a to b, all its heads and roles side by side)
// has n = max(1, ceil((b-a) / d)) items, and m <= n <= m + 1 with m = f(b) - f(a).  Its
// first m items have the numbers f(a) .. f(b) - 1, which no other sequence has; the
// one behind them, if there is one, has f(T) + s.  That makes f(T) + B numbers.  Those
// that stand for nothing are among the last (rows of no sequence apart), where the
// short items are: with them between the others 24 prompts in 18011 rows took 3 to 5 %
// longer (229 against 238 us in a captured graph).
// The n - 1 items of a cut sequence that have a state of their own are numbered
// f(a) .. as well, and so are the slots; behind these, at f(T) + f(a), lies the slot
// for the initial state of the chain's first item.
struct ScanPlan {
    int B, T, H, nroles;
    int packed;
    const int* cu;      // packed: [B+1] row offsets of the sequences
    int nfull, nseg;
    int seg_tokens;
    long long items;    // upper bound when packed
    // whether any chain can have several items
    SSD_HD bool cut() const { return packed ? T > seg_tokens : nseg > 1; }
    // packed: the numbers below f(T), over all heads and roles
    SSD_HD long long inner() const { return (long long)(T / seg_tokens) * H * nroles; }
    SSD_HD long long slots() const { return !cut() ? 0 : packed ? 2 * inner() : items - nfull; }
    // blocks of a state-only launch, and chains whose states are combined
    SSD_HD long long state_items() const { return packed ? inner() : items; }
    SSD_HD long long cut_chains() const { return packed ? inner() : (long long)B * H * nroles - nfull; }
};

struct ScanLaunch {
    ScanPlan plan;
    ScanRole role[kScanRoles];
    const float* decay;  // [H]
    float* states;       // [slots][K][V] of the items that are not their chain's last
    int* status;         // device status word
    int reset;           // the call's first kernel: its first block clears the status word
    bool bf16;
};

// The item `it` of a plan.
struct ScanItem {
    int role, seq, head;
    int seg, nseg;          // position among the chain's items, in scan order
    long long row0;         // first row of the sequence in the row dimension (0 when not packed)
    int batch;              // batch coordinate (0 when packed)
    int len;                // tokens of the sequence
    int t0, t1;             // this item's tokens [t0, t1) of the sequence
    // states: own (of an item that is not its chain's last), the one this item starts from,
    // and the chain's slot for the initial state, where its first item finds it (it may be read
    // late, when the final state, which may be the same memory, is written).  -1: not cut
    long long slot, slot_prev, slot_init;
    int valid;
};

// Number `number` (place hr among the heads and roles) as an item of packed sequence
// s, rows a to b: the last one with floor(a / seg_tokens) <= number, or s itself.
SSD_HD inline void packed_item(const ScanPlan& p, unsigned number, int hr, int s, int a, int b, ScanItem& r) {
    const int HR = p.H * p.nroles, whole = p.T / p.seg_tokens;
    const int first = a / p.seg_tokens, m = b / p.seg_tokens - first;
    const bool behind = number >= (unsigned)whole;
    r.seq = s;
    r.row0 = a;
    r.batch = 0;
    r.len = b - a;
    r.head = hr / p.nroles;
    r.role = hr - r.head * p.nroles;
    r.nseg = r.len <= p.seg_tokens ? 1 : (r.len - 1) / p.seg_tokens + 1;
    r.seg = behind ? m : (int)number - first;
    r.valid = r.seg < (behind ? r.nseg : m);  // else a number that stands for nothing
    if (!r.valid || r.nseg == 1) return;
    r.slot = (long long)(first + r.seg) * HR + hr;
    r.slot_init = ((long long)whole + first) * HR + hr;
    r.slot_prev = r.seg > 0 ? r.slot - HR : r.slot_init;
}

// The tokens of the item, given the direction of its role.
SSD_HD inline void scan_item_tokens(ScanItem& r, int seg_tokens, int reverse) {
    if (r.nseg == 1) {
        r.t0 = 0;
        r.t1 = r.len;
    } else {
        const int j = reverse ? r.nseg - 1 - r.seg : r.seg;
        r.t0 = j * seg_tokens;
        r.t1 = r.len - r.t0 > seg_tokens ? r.t0 + seg_tokens : r.len;  // (len may be near 2^31)
    }
}

#ifdef __CUDACC__
// The last of the B packed sequences with floor(a / seg_tokens) <= number, and its
// rows a and b; -1 if there is none.  Called by the 32 lanes of one warp, which look at
// 32 places at a time: B sequences take log33 B rounds.  Offsets that are no offsets
// (negative, beyond T, decreasing) are clamped, so that no row outside [0, T) and no slot
// outside the workspace is ever addressed.
__device__ inline int packed_offset(const ScanPlan& p, int s) { return min(max(p.cu[s], 0), p.T); }
__device__ inline int packed_sequence(const ScanPlan& p, unsigned number, int& a, int& b) {
    const int lane = threadIdx.x & 31;
    int lo = -1, hi = p.B, at_lo = 0, at_hi = packed_offset(p, p.B);
    while (hi - lo > 1) {
        const int step = (hi - lo + 32) / 33;
        const long long place = lo + (lane + 1LL) * step;
        const bool there = place < hi;
        const int s = there ? (int)place : hi;
        const int c = there ? packed_offset(p, s) : at_hi;
        const unsigned below = __ballot_sync(0xffffffffu, there && (unsigned)c / (unsigned)p.seg_tokens <= number);
        const int n = below == 0xffffffffu ? 32 : __ffs(~below) - 1;  // places in front that are
        const int next = __shfl_sync(0xffffffffu, s, n & 31), at_next = __shfl_sync(0xffffffffu, c, n & 31);
        const int last = __shfl_sync(0xffffffffu, s, (n + 31) & 31), at_last = __shfl_sync(0xffffffffu, c, (n + 31) & 31);
        if (n < 32) hi = next, at_hi = at_next;
        if (n > 0) lo = last, at_lo = at_last;
    }
    a = at_lo;
    b = max(at_hi, at_lo);
    return lo;
}
// Item `it` of a plan.  Called by the 32 lanes of one warp; the result is the same in
// every lane.
__device__ inline ScanItem scan_item(const ScanPlan& p, long long it) {
    ScanItem r;
    r.valid = 0;
    r.row0 = 0;
    r.slot = r.slot_prev = r.slot_init = -1;
    if (!p.packed) {
        // an item is a block of a grid: 32 bits hold it, and their divisions are short
        unsigned cr = (unsigned)it;
        int seg = 0, nseg = 1;
        if (it >= p.nfull) {
            const unsigned rest = cr - (unsigned)p.nfull, chain = rest / (unsigned)p.nseg;
            cr = (unsigned)p.nfull + chain;
            seg = (int)(rest - chain * (unsigned)p.nseg);
            nseg = p.nseg;
            r.slot = rest;
            r.slot_init = r.slot - seg + nseg - 1;
            r.slot_prev = seg > 0 ? r.slot - 1 : nseg > 1 ? r.slot_init : -1;
        }
        const unsigned hr = p.nroles == 1 ? cr : cr / (unsigned)p.nroles;
        r.role = (int)(cr - hr * (unsigned)p.nroles);
        r.seq = (int)(hr / (unsigned)p.H);
        r.head = (int)(hr - (unsigned)r.seq * (unsigned)p.H);
        r.batch = r.seq;
        r.len = p.T;
        r.seg = seg;
        r.nseg = nseg;
        r.valid = 1;
    } else {
        const unsigned HR = (unsigned)(p.H * p.nroles), number = (unsigned)it / HR;
        const unsigned whole = (unsigned)p.T / (unsigned)p.seg_tokens;
        int a, b, seq;
        if (number < whole) {
            seq = packed_sequence(p, number, a, b);
        } else {
            seq = (int)(number - whole);
            a = packed_offset(p, seq);
            b = max(packed_offset(p, seq + 1), a);
        }
        if (seq >= 0) packed_item(p, number, (int)((unsigned)it - number * HR), seq, a, b, r);
    }
    return r;
}
// exp(decay * n) as an unevaluated sum of two fp32 numbers: a long chain
// multiplies its state by the same factor at every chunk, and the error of one
// rounded factor would grow with the number of chunks the state remembers.
// Not inlined: a 64-bit exponential is long, and the scan's loops have to stay
// in the instruction cache.
static __device__ __noinline__ float2 decay_power(float decay, int n) {
    const double e = n == 0 ? 1.0 : exp((double)decay * n);
    const float hi = (float)e;
    return make_float2(hi, (float)(e - (double)hi));
}
#endif

#ifdef __CUDACC__
// Kernels of one call overlap at their ends: a kernel lets the next one's blocks start
// as soon as all of its own have (they take the places that its last ones leave, and
// make their tables), and a block waits, before it touches what an earlier kernel
// reads or writes, until all kernels before its own are done.  Some block of each
// kernel waits in any case, so that a kernel is never done before the earlier ones.
// (Gradients of 32768 x 2560 norms 104 -> 97 us, 24 packed prompts 172 -> 166.)
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// kernel<<<grid, block, smem, st>>>(args); behind: it follows a kernel of the same call
template <typename... P, typename... A>
cudaError_t launch_in_call(void (*kernel)(P...), unsigned grid, int block, size_t smem, cudaStream_t st, bool behind,
                           const A&... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid);
    c.blockDim = dim3((unsigned)block);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = at;
    c.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, args...);
}
#endif

// ---- launchers --------------------------------------------------------------
// CUDA cores, fp32 arithmetic: any sizes up to 256, any strides.  state_only:
// the states of the items that are not their chain's last, into `states`.
cudaError_t launch_scan_simt(const ScanLaunch& s, bool state_only, cudaStream_t st);
// Tensor cores (linear_tc.cu): bf16, sizes up to 128 and multiples of 8, rows
// on 16-byte boundaries.
struct ScanMaps { alignas(64) unsigned char map[kScanRoles][4][128]; };  // CUtensorMap of q, k, v and out
// the roles' maps; false: not for this kernel
bool scan_tc_maps(const ScanLaunch& s, ScanMaps& m);
cudaError_t launch_scan_tc(const ScanLaunch& s, const ScanMaps& m, bool state_only, cudaStream_t st);
// states in place: slot i from "built by item i from zero" to "after item i"
cudaError_t launch_scan_combine(const ScanLaunch& s, cudaStream_t st);
// out[row][g][d] = sum over the heads of group g of part[row][h][d]
cudaError_t launch_group_sum(const float* part, void* out, long long rows, int H, int G, int D, const int* cu, int B,
                             bool bf16, cudaStream_t st);

struct LinearStep {
    RowTensor q, k, v;
    int B, H, K, V;
    const float* decay;
    float scale;
    float* state;  // [B][H][K][V]
    void* y;       // [B][H][V]
    bool bf16;
};
cudaError_t launch_linear_step(const LinearStep& s, cudaStream_t st);

struct NormArgs {
    long long rows;
    int width, groups;
    bool bf16;
    const void* x;
    long long x_stride;
    const float* weight;  // or null
    const float* bias;    // or null
    const void* gate;     // or null
    long long gate_stride;
    float eps;
    void* y;
    float* stats;  // [rows][groups][2], or null
    // backward
    const void* dy;
    long long dy_stride;
    void* dx;
    float* dweight;  // or null
    float* dbias;    // or null
    void* dgate;
    float* part;  // [norm_backward_parts][2][width]
};
cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t st);
// rows of partial sums that the backward writes
int norm_backward_parts(long long rows, int width, int groups, bool bf16);
cudaError_t launch_layer_norm_backward(const NormArgs& a, cudaStream_t st);

}  // namespace ssd

// linear_api.cu -- the C ABI of linear attention with a decay for each head and
// of layer norm (declared in include/ssd.h): argument checks, workspace layout,
// how a call is cut into items, and the launches on the caller's stream.  No
// allocation happens here; every buffer belongs to the caller.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "common.cuh"
#include "kernels.h"
#include "linear.h"

namespace {

using ssd::RowTensor;
using ssd::ScanLaunch;
using ssd::ScanPlan;
using ssd::ScanRole;

constexpr size_t kAlign = 256;
constexpr size_t kCtrl = 256;  // status word
constexpr int kSMs = 148;
constexpr int kMaxDim = 256;

size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool on(const void* p, size_t a) { return p && ((uintptr_t)p % a) == 0; }
bool on_or_null(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
ssd_status status_of(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

// Where a call's chains are cut.  `at_once`: items that the GPU runs side by
// side.  Whole rounds of uncut chains come first.  The chains left over would
// leave part of the GPU idle for a whole chain's time, so they are cut into
// nseg items each where that is shorter, although a cut chain's k and v are
// read twice (state-only items first: about 0.6 of a full item's time).
// `start`, `launches`: an item's start and the two further launches, in units
// of one chunk.
void plan_rows(ScanPlan& p, int at_once, int chunk, double start, double launches) {
    const long long chains = (long long)p.B * p.H * p.nroles;
    const int nch = cdiv(p.T, chunk);
    const long long left = chains % at_once;
    int best = 1;
    double cost = nch + start;
    if (left > 0) {
        for (int s = 2; s <= nch && s <= 256; ++s) {
            const int per = cdiv(nch, s);
            const int n = cdiv(nch, per);
            const double c = (per + start) * (cdiv(left * n, at_once) + 0.6 * cdiv(left * (n - 1), at_once)) + launches;
            if (c < cost) {
                cost = c;
                best = s;
            }
        }
    }
    if (best == 1) {
        p.nfull = (int)chains;
        p.nseg = 1;
        p.seg_tokens = p.T;
        p.items = chains;
        return;
    }
    const int per = cdiv(nch, best);
    p.seg_tokens = per * chunk;
    p.nseg = cdiv(nch, per);
    p.nfull = (int)(chains - left);
    p.items = p.nfull + left * p.nseg;
}

// Packed sequences: their lengths are on the device, so every sequence is cut
// at the same distance, which gives about three items for each that runs at a
// time if the tokens are spread evenly, and never less than four chunks.
void plan_packed(ScanPlan& p, int at_once, int chunk, const int* cu) {
    const long long all = (long long)p.T * p.H * p.nroles;
    long long seg = all / (3LL * at_once) / chunk * chunk;
    if (seg < 4 * chunk) seg = 4 * chunk;
    if (seg > (1 << 30)) seg = 1 << 30;
    p.packed = 1;
    p.cu = cu;
    p.nfull = 0;
    p.nseg = 0;
    p.seg_tokens = (int)seg;
    p.items = ((long long)p.B + p.T / seg) * p.H * p.nroles;
}

ScanPlan make_plan(const ssd_linear_shape& s, int nroles, int vmax, bool tc, const int* cu) {
    ScanPlan p = {};
    p.B = s.B;
    p.T = s.T;
    p.H = s.H;
    p.nroles = nroles;
    // tensor cores: one block per SM; CUDA cores: two, of 64 state columns each
    const int tiles = cdiv(vmax, ssd::kSimtColumns);
    int at_once = tc ? kSMs : 2 * kSMs / tiles;
    // (CUDA cores: bounds every 128 tokens instead of 32 cost 52 against 33 us for 2 x 333
    // tokens of 8 heads; without the states' size in an item's start the gradients of 1 x 300
    // tokens, 24 heads, 128 x 128 took 173 us instead of 131)
    if (s.packed) plan_packed(p, at_once, tc ? ssd::kScanChunk : ssd::kSimtChunk, cu);
    else if (tc) plan_rows(p, at_once, ssd::kScanChunk, 1.5, 3.0);
    else plan_rows(p, at_once, ssd::kSimtChunk, 0.5 * s.K * s.V / 4096.0, 1.0);
    return p;
}

ssd_status check_linear(const ssd_linear_shape* s) {
    if (!s) return SSD_ERR_INVALID_ARG;
    if (s->B < 1 || s->T < 1 || s->H < 1 || s->G < 1 || s->K < 1 || s->V < 1) return SSD_ERR_INVALID_ARG;
    if (s->H % s->G != 0 || s->K > kMaxDim || s->V > kMaxDim) return SSD_ERR_INVALID_ARG;
    if (s->T > 0x7fffffff - 1024) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    if (s->packed != 0 && s->packed != 1) return SSD_ERR_INVALID_ARG;
    // the grids: items of up to three scans, up to four column tiles each
    if ((long long)s->B * s->H > 0x7fffffffLL / 12) return SSD_ERR_INVALID_ARG;
    if (s->packed && ((long long)s->B + s->T / 512) * s->H > 0x7fffffffLL / 12) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

// contiguous strides of [B][T][heads][d], for a tensor given without any
ssd_strides dense(const ssd_linear_shape& s, int heads, int d) {
    ssd_strides r;
    r.head = d;
    r.token = (long long)heads * d;
    r.batch = r.token * s.T;
    return r;
}
RowTensor tensor(const ssd_linear_shape& s, const void* p, const ssd_strides* st, int heads, int d) {
    const ssd_strides r = st ? *st : dense(s, heads, d);
    RowTensor t;
    t.p = p;
    t.batch = s.packed ? 0 : r.batch;
    t.token = r.token;
    t.head = r.head;
    t.share = s.H / heads;
    return t;
}
bool strides_ok(const ssd_strides* st) { return !st || (st->batch >= 0 && st->token >= 0 && st->head >= 0); }

int pad64(int d) { return d <= 64 ? 64 : 128; }

// rounded up over both ways of running it: which one serves a call depends on
// its strides and addresses too
size_t slots_bytes(const ssd_linear_shape& s, int nroles, int vmax, bool backward) {
    size_t most = 0;
    for (int tc = 0; tc < 2; ++tc) {
        for (int n = 1; n <= nroles; ++n) {
            if (!backward && n != nroles) continue;
            const ScanPlan p = make_plan(s, n, vmax, tc != 0, nullptr);
            const size_t b = (size_t)p.slots() * s.K * s.V * sizeof(float);
            if (b > most) most = b;
        }
    }
    return up(most);
}

long long rows_of(const ssd_linear_shape& s) { return s.packed ? s.T : (long long)s.B * s.T; }

// One scan launch: states of the cut chains, their combination, the outputs.
// maps: for the tensor cores, null = CUDA cores
cudaError_t run_scan(ScanLaunch& l, const ssd::ScanMaps* maps, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (l.plan.cut()) {
        e = maps ? ssd::launch_scan_tc(l, *maps, true, st) : ssd::launch_scan_simt(l, true, st);
        l.reset = 0;
        if (e == cudaSuccess) e = ssd::launch_scan_combine(l, st);
    }
    if (e == cudaSuccess) e = maps ? ssd::launch_scan_tc(l, *maps, false, st) : ssd::launch_scan_simt(l, false, st);
    l.reset = 0;
    return e;
}

}  // namespace

extern "C" {

size_t ssd_linear_workspace_size(const ssd_linear_shape* shape) {
    if (check_linear(shape) != SSD_OK) return 0;
    return kCtrl + slots_bytes(*shape, 1, shape->V, false);
}

ssd_status ssd_linear_attention(const ssd_linear_shape* shape, const void* q, const ssd_strides* q_strides,
                                const void* k, const ssd_strides* k_strides, const void* v,
                                const ssd_strides* v_strides, const float* decay, const int* cu_seqlens,
                                const float* initial_state, float scale, void* y, float* final_state,
                                void* workspace, size_t ws_bytes, ssd_stream stream) {
    if (check_linear(shape) != SSD_OK) return SSD_ERR_INVALID_ARG;
    const ssd_linear_shape& s = *shape;
    const size_t el = s.dtype == SSD_DTYPE_BF16 ? 2 : 4;
    if (!on(q, el) || !on(k, el) || !on(v, el) || !on(decay, 4) || !on(y, 16)) return SSD_ERR_INVALID_ARG;
    if (!strides_ok(q_strides) || !strides_ok(k_strides) || !strides_ok(v_strides)) return SSD_ERR_INVALID_ARG;
    if (s.packed ? !on(cu_seqlens, 4) : cu_seqlens != nullptr) return SSD_ERR_INVALID_ARG;
    if (!on_or_null(initial_state, 16) || !on_or_null(final_state, 16) || !isfinite(scale)) return SSD_ERR_INVALID_ARG;
    if (!on(workspace, kAlign) || ws_bytes < ssd_linear_workspace_size(shape)) return SSD_ERR_WORKSPACE;
    if (ssd::take_injected_failure()) return SSD_ERR_CUDA;
    ScanLaunch l = {};
    l.bf16 = s.dtype == SSD_DTYPE_BF16;
    l.decay = decay;
    l.status = (int*)workspace;
    l.reset = 1;
    l.states = (float*)((char*)workspace + kCtrl);
    ScanRole& r = l.role[0];
    r.q = tensor(s, q, q_strides, s.H, s.K);
    r.k = tensor(s, k, k_strides, s.G, s.K);
    r.v = tensor(s, v, v_strides, s.G, s.V);
    r.K = s.K;
    r.V = s.V;
    r.out = y;
    r.out_scale = scale;
    r.init = initial_state;
    r.init_k = s.V;
    r.init_v = 1;
    r.init_scale = 1.f;
    r.fin = final_state;
    r.fin_scale = 1.f;
    l.plan = make_plan(s, 1, s.V, true, cu_seqlens);
    ssd::ScanMaps maps;
    const bool tc = ssd::scan_tc_maps(l, maps);
    if (!tc) l.plan = make_plan(s, 1, s.V, false, cu_seqlens);
    return status_of(run_scan(l, tc ? &maps : nullptr, (cudaStream_t)stream));
}

ssd_status ssd_linear_attention_step(const ssd_linear_shape* shape, const void* q, const ssd_strides* q_strides,
                                     const void* k, const ssd_strides* k_strides, const void* v,
                                     const ssd_strides* v_strides, const float* decay, float scale, float* state,
                                     void* y, ssd_stream stream) {
    if (check_linear(shape) != SSD_OK || shape->T != 1 || shape->packed) return SSD_ERR_INVALID_ARG;
    const ssd_linear_shape& s = *shape;
    const size_t el = s.dtype == SSD_DTYPE_BF16 ? 2 : 4;
    if (!on(q, el) || !on(k, el) || !on(v, el) || !on(decay, 4) || !on(state, 16) || !on(y, el))
        return SSD_ERR_INVALID_ARG;
    if (!strides_ok(q_strides) || !strides_ok(k_strides) || !strides_ok(v_strides) || !isfinite(scale))
        return SSD_ERR_INVALID_ARG;
    if (ssd::take_injected_failure()) return SSD_ERR_CUDA;
    ssd::LinearStep p = {};
    p.q = tensor(s, q, q_strides, s.H, s.K);
    p.k = tensor(s, k, k_strides, s.G, s.K);
    p.v = tensor(s, v, v_strides, s.G, s.V);
    p.B = s.B;
    p.H = s.H;
    p.K = s.K;
    p.V = s.V;
    p.decay = decay;
    p.scale = scale;
    p.state = state;
    p.y = y;
    p.bf16 = s.dtype == SSD_DTYPE_BF16;
    return status_of(ssd::launch_linear_step(p, (cudaStream_t)stream));
}

size_t ssd_linear_backward_workspace_size(const ssd_linear_shape* shape) {
    if (check_linear(shape) != SSD_OK) return 0;
    const ssd_linear_shape& s = *shape;
    size_t n = kCtrl + slots_bytes(s, 3, s.K > s.V ? s.K : s.V, true);
    if (s.H != s.G) n += up((size_t)rows_of(s) * s.H * s.K * 4) + up((size_t)rows_of(s) * s.H * s.V * 4);
    return n;
}

ssd_status ssd_linear_attention_backward(const ssd_linear_shape* shape, const void* q, const ssd_strides* q_strides,
                                         const void* k, const ssd_strides* k_strides, const void* v,
                                         const ssd_strides* v_strides, const float* decay, const int* cu_seqlens,
                                         const float* initial_state, float scale, const void* dy, const float* dfinal,
                                         void* dq, void* dk, void* dv, float* dinit, void* workspace,
                                         size_t ws_bytes, ssd_stream stream) {
    if (check_linear(shape) != SSD_OK) return SSD_ERR_INVALID_ARG;
    const ssd_linear_shape& s = *shape;
    const size_t el = s.dtype == SSD_DTYPE_BF16 ? 2 : 4;
    if (!on(q, el) || !on(k, el) || !on(v, el) || !on(decay, 4) || !on(dy, 16) || !on(dq, 16) || !on(dk, 16) ||
        !on(dv, 16))
        return SSD_ERR_INVALID_ARG;
    if (!strides_ok(q_strides) || !strides_ok(k_strides) || !strides_ok(v_strides)) return SSD_ERR_INVALID_ARG;
    if (s.packed ? !on(cu_seqlens, 4) : cu_seqlens != nullptr) return SSD_ERR_INVALID_ARG;
    if (!on_or_null(initial_state, 16) || !on_or_null(dfinal, 16) || !on_or_null(dinit, 16)) return SSD_ERR_INVALID_ARG;
    // the adjoint state is kept without the factor `scale`: dfinal enters divided by it
    if (!isfinite(scale) || !isfinite(1.f / scale)) return SSD_ERR_INVALID_ARG;
    if (!on(workspace, kAlign) || ws_bytes < ssd_linear_backward_workspace_size(shape)) return SSD_ERR_WORKSPACE;
    if (ssd::take_injected_failure()) return SSD_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    const bool shared = s.H != s.G;
    ScanLaunch l = {};
    l.bf16 = s.dtype == SSD_DTYPE_BF16;
    l.decay = decay;
    l.status = (int*)workspace;
    l.reset = 1;
    l.states = (float*)((char*)workspace + kCtrl);
    const int vmax = s.K > s.V ? s.K : s.V;
    char* parts = (char*)workspace + kCtrl + slots_bytes(s, 3, vmax, true);
    float* dk_part = (float*)parts;
    float* dv_part = (float*)(parts + up((size_t)rows_of(s) * s.H * s.K * 4));
    const RowTensor tq = tensor(s, q, q_strides, s.H, s.K), tk = tensor(s, k, k_strides, s.G, s.K),
                    tv = tensor(s, v, v_strides, s.G, s.V), tdy = tensor(s, dy, nullptr, s.H, s.V);
    ScanRole a = {}, b = {}, c = {};
    // dq: forwards over (dy, v, k), from the transposed initial state
    a.q = tdy; a.k = tv; a.v = tk;
    a.K = s.V; a.V = s.K;
    a.out = dq;
    a.init = initial_state; a.init_k = 1; a.init_v = s.V; a.init_scale = 1.f;
    // dk: backwards over (v, dy, q), from the transposed gradient of the final state
    b.q = tv; b.k = tdy; b.v = tq;
    b.K = s.V; b.V = s.K;
    b.reverse = 1;
    b.out = shared ? (void*)dk_part : dk;
    b.out_f32 = shared;
    b.init = dfinal; b.init_k = 1; b.init_v = s.V; b.init_scale = 1.f / scale;
    // dv: backwards over (k, q, dy); its last state is the initial state's gradient
    c.q = tk; c.k = tq; c.v = tdy;
    c.K = s.K; c.V = s.V;
    c.reverse = 1;
    c.out = shared ? (void*)dv_part : dv;
    c.out_f32 = shared;
    c.init = dfinal; c.init_k = s.V; c.init_v = 1; c.init_scale = 1.f / scale;
    c.fin = dinit;
    c.fin_scale = scale;
    a.out_scale = b.out_scale = c.out_scale = scale;
    l.role[0] = a;
    l.role[1] = b;
    l.role[2] = c;
    l.plan = make_plan(s, 3, vmax, true, cu_seqlens);
    cudaError_t e;
    ssd::ScanMaps maps;
    if (!ssd::scan_tc_maps(l, maps)) {
        l.plan = make_plan(s, 3, vmax, false, cu_seqlens);
        e = run_scan(l, nullptr, st);
    } else if (pad64(s.K) == pad64(s.V)) {
        e = run_scan(l, &maps, st);
    } else {  // dq and dk have the state [V][K], dv has [K][V]: other tiles
        l.plan = make_plan(s, 2, vmax, true, cu_seqlens);
        e = run_scan(l, &maps, st);
        l.role[0] = c;
        memcpy(maps.map[0], maps.map[2], sizeof maps.map[0]);
        l.plan = make_plan(s, 1, vmax, true, cu_seqlens);
        if (e == cudaSuccess) e = run_scan(l, &maps, st);
    }
    if (shared) {
        if (e == cudaSuccess) e = ssd::launch_group_sum(dk_part, dk, rows_of(s), s.H, s.G, s.K, cu_seqlens, s.B,
                                                           l.bf16, st);
        if (e == cudaSuccess) e = ssd::launch_group_sum(dv_part, dv, rows_of(s), s.H, s.G, s.V, cu_seqlens, s.B,
                                                           l.bf16, st);
    }
    return status_of(e);
}

static ssd_status check_norm(const ssd_norm_shape* s) {
    if (!s || s->rows < 1 || s->width < 1 || s->groups < 1 || s->width % s->groups != 0) return SSD_ERR_INVALID_ARG;
    if (s->width / s->groups > 16384 || s->rows > (1LL << 40)) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

static ssd::NormArgs norm_args(const ssd_norm_shape* s) {
    ssd::NormArgs a = {};
    a.rows = s->rows;
    a.width = s->width;
    a.groups = s->groups;
    a.bf16 = s->dtype == SSD_DTYPE_BF16;
    return a;
}

ssd_status ssd_layer_norm(const ssd_norm_shape* shape, const void* x, long long x_stride, const float* weight,
                          const float* bias, const void* gate, long long gate_stride, float eps, void* y,
                          float* stats, ssd_stream stream) {
    if (check_norm(shape) != SSD_OK) return SSD_ERR_INVALID_ARG;
    const size_t el = shape->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    if (!on(x, el) || !on(y, el) || !on_or_null(gate, el) || !on_or_null(weight, 4) || !on_or_null(bias, 4) ||
        !on_or_null(stats, 8) || x_stride < 0 || gate_stride < 0)
        return SSD_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !isfinite(eps)) return SSD_ERR_INVALID_ARG;
    if (ssd::take_injected_failure()) return SSD_ERR_CUDA;
    ssd::NormArgs a = norm_args(shape);
    a.x = x;
    a.x_stride = x_stride;
    a.weight = weight;
    a.bias = bias;
    a.gate = gate;
    a.gate_stride = gate_stride;
    a.eps = eps;
    a.y = y;
    a.stats = stats;
    return status_of(ssd::launch_layer_norm(a, (cudaStream_t)stream));
}

size_t ssd_layer_norm_backward_workspace_size(const ssd_norm_shape* shape) {
    if (check_norm(shape) != SSD_OK) return 0;
    const int parts = ssd::norm_backward_parts(shape->rows, shape->width, shape->groups,
                                               shape->dtype == SSD_DTYPE_BF16);
    return up((size_t)parts * 2 * shape->width * sizeof(float));
}

ssd_status ssd_layer_norm_backward(const ssd_norm_shape* shape, const void* x, long long x_stride,
                                   const float* weight, const float* bias, const void* gate,
                                   long long gate_stride, const void* dy, long long dy_stride, const float* stats,
                                   void* dx, float* dweight, float* dbias, void* dgate, void* workspace,
                                   size_t ws_bytes, ssd_stream stream) {
    if (check_norm(shape) != SSD_OK) return SSD_ERR_INVALID_ARG;
    const size_t el = shape->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    if (!on(x, el) || !on(dy, el) || !on(dx, el) || !on(stats, 8) || !on_or_null(gate, el) ||
        !on_or_null(weight, 4) || !on_or_null(bias, 4) || !on_or_null(dweight, 4) || !on_or_null(dbias, 4) ||
        x_stride < 0 || gate_stride < 0 || dy_stride < 0)
        return SSD_ERR_INVALID_ARG;
    if (gate ? !on(dgate, el) : dgate != nullptr) return SSD_ERR_INVALID_ARG;
    const bool sums = dweight || dbias;
    if (sums && (!on(workspace, kAlign) || ws_bytes < ssd_layer_norm_backward_workspace_size(shape)))
        return SSD_ERR_WORKSPACE;
    if (ssd::take_injected_failure()) return SSD_ERR_CUDA;
    ssd::NormArgs a = norm_args(shape);
    a.x = x;
    a.x_stride = x_stride;
    a.weight = weight;
    a.bias = bias;
    a.gate = gate;
    a.gate_stride = gate_stride;
    a.stats = const_cast<float*>(stats);
    a.dy = dy;
    a.dy_stride = dy_stride;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dgate = dgate;
    a.part = sums ? (float*)workspace : nullptr;
    return status_of(ssd::launch_layer_norm_backward(a, (cudaStream_t)stream));
}

}  // extern "C"

// C ABI of the operators around a mixing layer: argument validation.  As in kda_api.cu, a
// rejected call enqueues nothing.
#include <climits>
#include <cmath>

#include "kda_block.cuh"

namespace {

using namespace kda;

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool known(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
unsigned bytes_of(kda_dtype t) { return t == KDA_BF16 ? 2u : 4u; }

// Required pointers (null only for an empty call), and ones that may be null.
kda_status check_ptrs(bool empty, unsigned align, std::initializer_list<const void*> required,
                      std::initializer_list<const void*> optional) {
    for (const void* p : required) {
        if (!p && !empty) return KDA_ERR_INVALID_ARG;
        if (!aligned(p, align)) return KDA_ERR_ALIGNMENT;
    }
    for (const void* p : optional)
        if (!aligned(p, align)) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

kda_status check_ws(size_t need, const void* ws, size_t bytes) {
    if (!ws || bytes < need) return KDA_ERR_WORKSPACE;
    return aligned(ws, 256) ? KDA_OK : KDA_ERR_ALIGNMENT;
}

// ---- the gated recurrence ----

// What a row or element index of the kernels may reach.
constexpr long long kMaxRows = 1LL << 30;

kda_status check_scan(const kda_scan_dims* d, const int* cu, int nseq) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (!known(d->dtype)) return KDA_ERR_INVALID_ARG;
    if (d->B < 0 || d->T < 0 || d->C <= 0) return KDA_ERR_SHAPE;
    if (cu && (d->B != 1 || nseq < 1)) return KDA_ERR_SHAPE;
    if (d->B > 65535 || nseq > 65535 || (long long)d->B * d->T >= kMaxRows || d->C >= kMaxRows)
        return KDA_ERR_UNSUPPORTED;
    // a token's channels do not reach into the next token's; strides of a dimension of one are
    // not used
    const long long st[2][2] = {{d->x_batch, d->x_token}, {d->g_batch, d->g_token}};
    for (auto& s : st)
        if ((d->T > 1 && s[1] < d->C) || (d->B > 1 && s[0] < d->C)) return KDA_ERR_SHAPE;
    return aligned(cu, 4) ? KDA_OK : KDA_ERR_ALIGNMENT;
}

ScanArgs scan_args(const kda_scan_dims& d, const void* x, const void* g, const float* h0,
                   const int* cu, int nseq) {
    ScanArgs a = {};
    a.B = d.B;
    a.T = d.T;
    a.C = d.C;
    a.tied = d.tied != 0;
    a.x_batch = d.x_batch;
    a.x_token = d.x_token;
    a.g_batch = d.g_batch;
    a.g_token = d.g_token;
    a.x = x;
    a.g = g;
    a.h0 = h0;
    a.cu = cu;
    a.nseq = nseq;
    return a;
}

// No tokens at all: what enters leaves.
kda_status pass_on(const kda_scan_dims& d, const int* cu, int nseq, const float* from, float* to,
                   cudaStream_t s) {
    if (!to) return KDA_OK;
    const size_t n = (size_t)(cu ? nseq : d.B) * d.C * sizeof(float);
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, n, cudaMemcpyDeviceToDevice, s)
                               : cudaMemsetAsync(to, 0, n, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// ---- the norms ----

kda_status check_gated(const kda_gated_norm_dims* d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (!known(d->dtype) || !known(d->w_dtype)) return KDA_ERR_INVALID_ARG;
    if (d->gate != KDA_GATE_SIGMOID && d->gate != KDA_GATE_SILU) return KDA_ERR_INVALID_ARG;
    if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return KDA_ERR_INVALID_ARG;
    if (d->T < 0 || d->H <= 0 || d->D <= 0) return KDA_ERR_SHAPE;
    if (d->D > block::kMaxWidth || (long long)d->T * d->H >= kMaxRows) return KDA_ERR_UNSUPPORTED;
    const long long row = (long long)d->H * d->D;
    if (d->T > 1 && (d->x_stride < row || d->gate_stride < row)) return KDA_ERR_SHAPE;
    return KDA_OK;
}

GatedArgs gated_args(const kda_gated_norm_dims& d, const void* x, const void* z, const void* w) {
    GatedArgs a = {};
    a.T = d.T;
    a.H = d.H;
    a.D = d.D;
    a.act = d.gate;
    a.eps = d.eps;
    a.x_stride = d.x_stride;
    a.z_stride = d.gate_stride;
    a.x = x;
    a.z = z;
    a.w = {w, d.w_dtype == KDA_BF16};
    return a;
}

kda_status check_add(const kda_add_norm_dims* d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (!known(d->dtype) || !known(d->res_dtype) || !known(d->w_dtype)) return KDA_ERR_INVALID_ARG;
    if (!(d->eps > 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->alpha))
        return KDA_ERR_INVALID_ARG;
    if (d->T < 0 || d->D <= 0) return KDA_ERR_SHAPE;
    if (d->D > block::kMaxWidth || d->T >= kMaxRows) return KDA_ERR_UNSUPPORTED;
    if (d->res_dtype == KDA_BF16 && d->dtype == KDA_F32) return KDA_ERR_UNSUPPORTED;
    if (d->T > 1 && (d->r_stride < d->D || d->x_stride < d->D)) return KDA_ERR_SHAPE;
    return KDA_OK;
}

int add_type(const kda_add_norm_dims& d) {
    return d.dtype == KDA_F32 ? 1 : d.res_dtype == KDA_F32 ? 2 : 0;
}

AddArgs add_args(const kda_add_norm_dims& d, const void* r, const void* x, const void* av,
                 const void* w) {
    AddArgs a = {};
    a.T = d.T;
    a.D = d.D;
    a.eps = d.eps;
    a.alpha = d.alpha;
    a.r_stride = d.r_stride;
    a.x_stride = d.x_stride;
    a.r = r;
    a.x = x;
    a.av = {av, d.w_dtype == KDA_BF16};
    a.w = {w, d.w_dtype == KDA_BF16};
    return a;
}

kda_status zero(float* p, int n, cudaStream_t s) {
    return !p || cudaMemsetAsync(p, 0, n * sizeof(float), s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status check_pack(long long rows, int D, kda_dtype t) {
    if (!known(t)) return KDA_ERR_INVALID_ARG;
    if (rows < 0 || D <= 0) return KDA_ERR_SHAPE;
    // the element count stays far from what 64 bits hold
    return rows > (1LL << 40) / D ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_gated_scan_fwd(const kda_scan_dims* d, const int* cu, int nseq, const void* x,
                              const void* g, const float* h0, void* o, float* ht, float* states,
                              void* stream) {
    kda_status st = check_scan(d, cu, nseq);
    if (st != KDA_OK) return st;
    const bool empty = d->B == 0 || d->T == 0;
    if ((st = check_ptrs(empty, bytes_of(d->dtype), {x, g}, {o})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, 4, {}, {h0, ht, states})) != KDA_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) return d->B == 0 ? KDA_OK : pass_on(*d, cu, nseq, h0, ht, s);
    if (!o && !ht && !states) return KDA_OK;
    ScanArgs a = scan_args(*d, x, g, h0, cu, nseq);
    a.o = o;
    a.ht = ht;
    a.states = states;
    return scan_fwd_launch(a, d->dtype == KDA_BF16, s);
}

kda_status kda_gated_scan_bwd(const kda_scan_dims* d, const int* cu, int nseq, const void* x,
                              const void* g, const float* h0, const float* states,
                              const void* dout, const float* dht, void* dx, void* dg, float* dh0,
                              void* stream) {
    kda_status st = check_scan(d, cu, nseq);
    if (st != KDA_OK) return st;
    const bool empty = d->B == 0 || d->T == 0;
    if ((st = check_ptrs(empty, bytes_of(d->dtype), {x, g, dout, dx, dg}, {})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, 4, {states}, {h0, dht, dh0})) != KDA_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) return d->B == 0 ? KDA_OK : pass_on(*d, cu, nseq, dht, dh0, s);
    ScanArgs a = scan_args(*d, x, g, h0, cu, nseq);
    a.states = const_cast<float*>(states);
    a.dout = dout;
    a.dht = dht;
    a.dx = dx;
    a.dg = dg;
    a.dh0 = dh0;
    return scan_bwd_launch(a, d->dtype == KDA_BF16, s);
}

kda_status kda_gated_scan_step(const kda_scan_dims* d, const void* x, const void* g,
                               const float* state, float* new_state, void* o, void* stream) {
    if (!d) return KDA_ERR_INVALID_ARG;
    kda_scan_dims t = *d;
    t.T = 1;
    kda_status st = check_scan(&t, nullptr, 0);
    if (st != KDA_OK) return st;
    if ((st = check_ptrs(d->B == 0, bytes_of(d->dtype), {x, g, o}, {})) != KDA_OK) return st;
    if ((st = check_ptrs(d->B == 0, 4, {state, new_state}, {})) != KDA_OK) return st;
    if (d->B == 0) return KDA_OK;
    return scan_step_launch(d->B, d->C, d->dtype == KDA_BF16, d->tied != 0, x, d->x_batch, g,
                            d->g_batch, state, new_state, o, static_cast<cudaStream_t>(stream));
}

kda_status kda_gated_norm_fwd(const kda_gated_norm_dims* d, const void* x, const void* gate,
                              const void* w, void* y, void* x_codes, unsigned char* x_scales,
                              void* gate_codes, unsigned char* gate_scales, void* stream) {
    kda_status st = check_gated(d);
    if (st != KDA_OK) return st;
    const bool empty = d->T == 0;
    if ((st = check_ptrs(empty, bytes_of(d->dtype), {x, gate, y}, {})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, bytes_of(d->w_dtype), {}, {w})) != KDA_OK) return st;
    // kept or not, all four together
    const int kept = !!x_codes + !!x_scales + !!gate_codes + !!gate_scales;
    if (kept != 0 && kept != 4 && !empty) return KDA_ERR_INVALID_ARG;
    if (empty) return KDA_OK;
    GatedArgs a = gated_args(*d, x, gate, w);
    a.y = y;
    a.xc = static_cast<uint8_t*>(x_codes);
    a.xs = x_scales;
    a.zc = static_cast<uint8_t*>(gate_codes);
    a.zs = gate_scales;
    return gated_norm_fwd_launch(a, d->dtype == KDA_BF16, static_cast<cudaStream_t>(stream));
}

size_t kda_gated_norm_workspace_bytes(const kda_gated_norm_dims* d) {
    return check_gated(d) == KDA_OK && d->T > 0 ? gated_norm_ws_bytes(d->T, d->H, d->D) : 0;
}

kda_status kda_gated_norm_bwd(const kda_gated_norm_dims* d, const void* x,
                              const unsigned char* x_scales, const void* gate,
                              const unsigned char* gate_scales, const void* w, const void* dy,
                              void* dx, void* dgate, float* dw, void* ws, size_t ws_bytes,
                              void* stream) {
    kda_status st = check_gated(d);
    if (st != KDA_OK) return st;
    const bool empty = d->T == 0, packed = x_scales || gate_scales;
    if (packed && !(x_scales && gate_scales) && !empty) return KDA_ERR_INVALID_ARG;
    if ((st = check_ptrs(empty, packed ? 1 : bytes_of(d->dtype), {x, gate}, {})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, bytes_of(d->dtype), {dy, dx, dgate}, {})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, bytes_of(d->w_dtype), {}, {w})) != KDA_OK) return st;
    if (!aligned(dw, 4)) return KDA_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) return zero(dw, d->D, s);
    if (dw && (st = check_ws(gated_norm_ws_bytes(d->T, d->H, d->D), ws, ws_bytes)) != KDA_OK) return st;
    GatedArgs a = gated_args(*d, x, gate, w);
    if (packed) {
        a.xc = static_cast<uint8_t*>(const_cast<void*>(x));
        a.zc = static_cast<uint8_t*>(const_cast<void*>(gate));
        a.xs = const_cast<uint8_t*>(x_scales);
        a.zs = const_cast<uint8_t*>(gate_scales);
    }
    a.dy = dy;
    a.dx = dx;
    a.dz = dgate;
    a.dw = dw;
    a.part = static_cast<float*>(ws);
    return gated_norm_bwd_launch(a, d->dtype == KDA_BF16, s);
}

kda_status kda_add_norm_fwd(const kda_add_norm_dims* d, const void* r, const void* x,
                            const void* alpha, const void* w, void* r_out, void* y, void* stream) {
    kda_status st = check_add(d);
    if (st != KDA_OK) return st;
    const bool empty = d->T == 0;
    if ((st = check_ptrs(empty, bytes_of(d->res_dtype), {r}, {r_out})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, bytes_of(d->dtype), {y}, {x})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, bytes_of(d->w_dtype), {}, {alpha, w})) != KDA_OK) return st;
    if (!empty && x && !r_out) return KDA_ERR_INVALID_ARG;
    if (empty) return KDA_OK;
    AddArgs a = add_args(*d, r, x, alpha, w);
    a.r_out = r_out;
    a.y = y;
    return add_norm_fwd_launch(a, add_type(*d), static_cast<cudaStream_t>(stream));
}

size_t kda_add_norm_workspace_bytes(const kda_add_norm_dims* d) {
    return check_add(d) == KDA_OK && d->T > 0 ? add_norm_ws_bytes(d->T, d->D) : 0;
}

kda_status kda_add_norm_bwd(const kda_add_norm_dims* d, const void* r, const void* x,
                            const void* alpha, const void* w, const void* dy, const void* dr,
                            void* dres, void* dx, float* dw, float* dalpha, void* ws,
                            size_t ws_bytes, void* stream) {
    kda_status st = check_add(d);
    if (st != KDA_OK) return st;
    const bool empty = d->T == 0;
    if ((st = check_ptrs(empty, bytes_of(d->res_dtype), {r, dres}, {dr})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, bytes_of(d->dtype), {dy}, {x, dx})) != KDA_OK) return st;
    if ((st = check_ptrs(empty, bytes_of(d->w_dtype), {}, {alpha, w})) != KDA_OK) return st;
    if (!aligned(dw, 4) || !aligned(dalpha, 4)) return KDA_ERR_ALIGNMENT;
    if (dalpha && !x && !empty) return KDA_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) return (st = zero(dw, d->D, s)) != KDA_OK ? st : zero(dalpha, d->D, s);
    if ((dw || dalpha) && (st = check_ws(add_norm_ws_bytes(d->T, d->D), ws, ws_bytes)) != KDA_OK)
        return st;
    AddArgs a = add_args(*d, r, x, alpha, w);
    a.dy = dy;
    a.dr = dr;
    a.dres = dres;
    a.dx = dx;
    a.dw = dw;
    a.da = dalpha;
    a.part = static_cast<float*>(ws);
    return add_norm_bwd_launch(a, add_type(*d), s);
}

kda_status kda_pack8(const void* x, kda_dtype dtype, long long rows, int D, long long x_stride,
                     void* codes, unsigned char* scales, void* stream) {
    kda_status st = check_pack(rows, D, dtype);
    if (st != KDA_OK) return st;
    if (rows > 1 && x_stride < D) return KDA_ERR_SHAPE;
    if ((st = check_ptrs(rows == 0, bytes_of(dtype), {x}, {})) != KDA_OK) return st;
    if ((st = check_ptrs(rows == 0, 1, {codes, scales}, {})) != KDA_OK) return st;
    if (rows == 0) return KDA_OK;
    return pack8_launch(x, dtype == KDA_BF16, rows, D, x_stride, static_cast<uint8_t*>(codes), scales,
                        static_cast<cudaStream_t>(stream));
}

kda_status kda_unpack8(const void* codes, const unsigned char* scales, long long rows, int D,
                       void* x, kda_dtype dtype, void* stream) {
    kda_status st = check_pack(rows, D, dtype);
    if (st != KDA_OK) return st;
    if ((st = check_ptrs(rows == 0, bytes_of(dtype), {x}, {})) != KDA_OK) return st;
    if ((st = check_ptrs(rows == 0, 1, {codes, scales}, {})) != KDA_OK) return st;
    if (rows == 0) return KDA_OK;
    return unpack8_launch(static_cast<const uint8_t*>(codes), scales, rows, D, x, dtype == KDA_BF16,
                          static_cast<cudaStream_t>(stream));
}

}  // extern "C"

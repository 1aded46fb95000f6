// Rotary positions of queries and keys (and values laid out beside them).
//
// Pair (x0, x1) number i of a head at position p turns by a = p f_i:
//   y0 = m (x0 cos a - x1 sin a),  y1 = m (x1 cos a + x0 sin a),
// and by -a in the transposed map (the gradient).  fp32 arithmetic, one
// rounding to the tensor's type at the store.
//
// Bound by HBM: every element is read once and written once.  A thread owns
// one token's 16 elements of a head (8 pairs: two 16-byte vectors in 16-bit
// types) and walks over heads, so a pair's angle, cosine and sine are
// computed once per token and thread and not once per head, with four heads'
// loads in flight.  A warp covers 4 tokens (d = 128): each of its loads
// touches whole 128-byte lines in both the head-major and the token-major
// layout.
// Measured: 65,536 tokens x 32 heads of 128, bf16, read token-major, written
// head-major: 170 us for 1.07 GB, 97% of the copy rate.  A decode step's
// queries (8 x 32 heads) take 4.2 us a call, bound by the launch.
#include <math.h>

#include <algorithm>
#include <new>

#include "rope.cuh"

namespace duo {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // heads whose loads are in flight

template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int UPH = D / 16;   // units per head
    // a programmatic dependent: nothing is read or written before what
    // precedes this launch has completed
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t item = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / UPH;
    const int u = threadIdx.x % UPH;
    if (item >= int64_t(p.B) * p.n) return;
    const int b = int(item / p.n), i = int(item - int64_t(b) * p.n);
    if (p.n_new && i >= p.n_new[b]) return;
    const RopeUnit unit = rope_unit(p.table, u);
    const int h0 = blockIdx.y * p.heads_per_thread;
    const int h1 = min(h0 + p.heads_per_thread, p.first_head[3]);

    float c[8], s[8];
    if (unit.rotates) {
        const int pos = p.per_token ? p.positions[item] : int(uint32_t(p.positions[b]) + uint32_t(i));
        rope_angles(p.table, u, pos, p.sign, c, s);
    }
    for (int h = h0; h < h1; h += kUnroll) {
        Vec8<T> v[kUnroll][2];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (h + k >= h1) break;
            const int w = (h + k >= p.first_head[1]) + (h + k >= p.first_head[2]);
            const RopeTensor& t = p.t[w];
            const T* x = static_cast<const T*>(t.in) + b * t.is_b + (h + k - p.first_head[w]) * t.is_h + i * t.is_t;
            v[k][0].load(x + unit.e0);
            v[k][1].load(x + unit.e1);
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (h + k >= h1) break;
            const int w = (h + k >= p.first_head[1]) + (h + k >= p.first_head[2]);
            const RopeTensor& t = p.t[w];
            T* y = static_cast<T*>(t.out) + b * t.os_b + (h + k - p.first_head[w]) * t.os_h + i * t.os_t;
            if (unit.rotates && t.rotate) {
                float x[16];
                widen(v[k][0], x);
                widen(v[k][1], x + 8);
                rope_rotate<HALF>(x, c, s);
                narrow(v[k][0], x);
                narrow(v[k][1], x + 8);
            }
            v[k][0].store(y + unit.e0);
            v[k][1].store(y + unit.e1);
        }
    }
}

template <typename T, int D>
cudaError_t launch_typed(const RopeParams& p, const cudaLaunchConfig_t& cfg) {
    return p.table.half ? cudaLaunchKernelEx(&cfg, rope_kernel<T, D, true>, p)
                        : cudaLaunchKernelEx(&cfg, rope_kernel<T, D, false>, p);
}

template <typename T>
cudaError_t launch_dim(const RopeParams& p, int d, const cudaLaunchConfig_t& cfg) {
    return d == 128 ? launch_typed<T, 128>(p, cfg) : launch_typed<T, 64>(p, cfg);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p0, int dtype, int head_dim, int num_sms, cudaStream_t s) {
    RopeParams p = p0;
    const int heads = p.first_head[3];
    const int64_t threads = int64_t(p.B) * p.n * (head_dim / 16);
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    // heads per thread: as many as leave a full wave of threads
    int hpt = 1;
    while (hpt < 16 && hpt < heads && threads * ((heads + 2 * hpt - 1) / (2 * hpt)) >= int64_t(num_sms) * 2048) hpt *= 2;
    // blockIdx.y stays within the grid's limit
    while ((heads + hpt - 1) / hpt > 65535) hpt *= 2;
    p.heads_per_thread = hpt;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks), unsigned((heads + hpt - 1) / hpt));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (dtype == DUO_BF16)
        e = launch_dim<__nv_bfloat16>(p, head_dim, cfg);
    else if (dtype == DUO_FP16)
        e = launch_dim<__half>(p, head_dim, cfg);
    else
        e = launch_dim<float>(p, head_dim, cfg);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace duo

// ------------------------------------------------------------------ the plan
namespace {

// Angles per position of every pair, from the description alone.
int make_angles(const duo_rope_desc& d, double* f, double* magnitude) {
    const double two_pi = 6.283185307179586476925286766559;
    const int pairs = d.rot_dim / 2;
    const double rot = d.rot_dim, s = d.factor, L = d.original_len;
    double theta = d.theta;
    if (d.scaling == DUO_ROPE_NTK) theta *= pow(s, rot / (rot - 2.0));
    for (int i = 0; i < pairs; ++i) f[i] = pow(theta, -2.0 * i / rot);
    *magnitude = 1.0;
    switch (d.scaling) {
        case DUO_ROPE_LINEAR:
            for (int i = 0; i < pairs; ++i) f[i] /= s;
            break;
        case DUO_ROPE_YARN: {
            const double slow = d.low > 0 ? d.low : 1.0, fast = d.high > 0 ? d.high : 32.0;
            if (!(fast > slow)) return DUO_ERR_INVALID_ARG;
            // the pair that makes t turns over the original length
            const auto pair_of = [&](double t) { return rot * log(L / (t * two_pi)) / (2.0 * log(theta)); };
            const double lo = std::max(floor(pair_of(fast)), 0.0), hi = std::min(ceil(pair_of(slow)), rot - 1.0);
            for (int i = 0; i < pairs; ++i) {
                const double r = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
                f[i] = f[i] * (1.0 - r) + f[i] / s * r;
            }
            if (s > 1.0) *magnitude = 0.1 * log(s) + 1.0;
            break;
        }
        case DUO_ROPE_BANDS: {
            const double low = d.low > 0 ? d.low : 1.0, high = d.high > 0 ? d.high : 4.0;
            if (!(high > low)) return DUO_ERR_INVALID_ARG;
            for (int i = 0; i < pairs; ++i) {
                const double r = std::min(std::max((L * f[i] / two_pi - low) / (high - low), 0.0), 1.0);
                f[i] = f[i] / s * (1.0 - r) + f[i] * r;
            }
            break;
        }
        case DUO_ROPE_FACTORS:
            for (int i = 0; i < pairs; ++i) f[i] /= d.pair_factors[i];
            break;
        default:
            break;
    }
    if (d.magnitude > 0) *magnitude = d.magnitude;
    for (int i = 0; i < pairs; ++i)
        if (!(f[i] >= 0.0) || !(f[i] < 1e6)) return DUO_ERR_INVALID_ARG;
    return DUO_OK;
}

bool positive(double x) { return x > 0.0 && x < 1e300; }

}  // namespace

extern "C" {

int duo_rope_create(const duo_rope_desc* d, duo_rope** out) {
    if (!d || !out) return DUO_ERR_INVALID_ARG;
    *out = nullptr;
    if (d->head_dim != 64 && d->head_dim != 128) return DUO_ERR_UNSUPPORTED;
    if (d->rot_dim < 16 || d->rot_dim > d->head_dim) return DUO_ERR_INVALID_ARG;
    if (d->rot_dim % 16 != 0) return DUO_ERR_UNSUPPORTED;
    if (d->layout != DUO_ROPE_HALF && d->layout != DUO_ROPE_INTERLEAVED) return DUO_ERR_INVALID_ARG;
    if (d->scaling < DUO_ROPE_NONE || d->scaling > DUO_ROPE_FACTORS) return DUO_ERR_INVALID_ARG;
    if (!(d->theta > 1.0) || !positive(d->theta)) return DUO_ERR_INVALID_ARG;
    const bool needs_factor = d->scaling != DUO_ROPE_NONE && d->scaling != DUO_ROPE_FACTORS;
    const bool needs_len = d->scaling == DUO_ROPE_YARN || d->scaling == DUO_ROPE_BANDS;
    if (needs_factor && (!(d->factor >= 1.0) || !positive(d->factor))) return DUO_ERR_INVALID_ARG;
    if (needs_len && (!positive(d->original_len) || !(d->low >= 0.0) || !(d->high >= 0.0) || d->low > 1e6 ||
                      d->high > 1e6))
        return DUO_ERR_INVALID_ARG;
    if (!(d->magnitude >= 0.0) || !(d->magnitude < 1e30)) return DUO_ERR_INVALID_ARG;
    if (d->scaling == DUO_ROPE_FACTORS) {
        if (!d->pair_factors) return DUO_ERR_INVALID_ARG;
        for (int i = 0; i < d->rot_dim / 2; ++i)
            if (!positive(d->pair_factors[i])) return DUO_ERR_INVALID_ARG;
    }
    duo_rope* r = new (std::nothrow) duo_rope();
    if (!r) return DUO_ERR_INVALID_ARG;
    r->desc = *d;
    const int rc = make_angles(*d, r->angle, &r->magnitude);
    r->desc.pair_factors = nullptr;
    if (rc) {
        delete r;
        return rc;
    }
    for (int i = 0; i < d->rot_dim / 2; ++i) {
        const double turns = r->angle[i] / 6.283185307179586476925286766559;
        // the fraction of a turn in units of 2^-64, from the 53 bits that it has
        r->turn[i] = uint64_t(ldexp(turns - floor(turns), 64));
    }
    *out = r;
    return DUO_OK;
}

int duo_rope_free(duo_rope* rope) {
    delete rope;
    return DUO_OK;
}

int duo_rope_frequencies(const duo_rope* rope, double* angle, double* magnitude) {
    if (!rope || !angle || !magnitude) return DUO_ERR_INVALID_ARG;
    for (int i = 0; i < rope->desc.rot_dim / 2; ++i) angle[i] = rope->angle[i];
    *magnitude = rope->magnitude;
    return DUO_OK;
}

int duo_rope_apply(const duo_rope* rope, int32_t dtype, int32_t transpose, int32_t batch, int32_t n,
                   const duo_rope_tensor* tensors, int32_t num_tensors, const int32_t* positions, int32_t per_token,
                   const int32_t* n_new, duo_stream_t stream) {
    if (!rope || !tensors || num_tensors < 1 || num_tensors > 3 || batch < 0 || n < 0) return DUO_ERR_INVALID_ARG;
    if (dtype != DUO_BF16 && dtype != DUO_FP16 && dtype != DUO_FP32) return DUO_ERR_INVALID_ARG;
    const int64_t vec = dtype == DUO_FP32 ? 4 : 8;   // elements of 16 bytes
    duo::RopeParams p = {};
    int heads = 0;
    for (int k = 0; k < 3; ++k) {
        p.first_head[k] = heads;
        if (k >= num_tensors) continue;
        const duo_rope_tensor& t = tensors[k];
        if (t.heads < 1 || t.heads > (1 << 20)) return DUO_ERR_INVALID_ARG;
        heads += t.heads;
    }
    p.first_head[3] = heads;
    if (batch == 0 || n == 0) return DUO_OK;
    if (!positions) return DUO_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(positions) & 3) || (reinterpret_cast<uintptr_t>(n_new) & 3))
        return DUO_ERR_ALIGNMENT;
    for (int k = 0; k < num_tensors; ++k) {
        const duo_rope_tensor& t = tensors[k];
        if (!t.in || !t.out) return DUO_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(t.in) & 15) || (reinterpret_cast<uintptr_t>(t.out) & 15))
            return DUO_ERR_ALIGNMENT;
        for (int j = 0; j < 3; ++j)
            if (t.in_stride[j] % vec != 0 || t.out_stride[j] % vec != 0) return DUO_ERR_ALIGNMENT;
        p.t[k] = duo::RopeTensor{t.in, t.out, t.in_stride[0], t.in_stride[1], t.in_stride[2],
                                 t.out_stride[0], t.out_stride[1], t.out_stride[2], t.rotate != 0};
    }
    p.B = batch;
    p.n = n;
    p.positions = positions;
    p.per_token = per_token != 0;
    p.n_new = n_new;
    p.sign = transpose ? -1.f : 1.f;
    p.table = duo::rope_table(rope);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return DUO_ERR_CUDA;
    return duo::launch_rope(p, dtype, rope->desc.head_dim, sms, stream) == cudaSuccess ? DUO_OK : DUO_ERR_CUDA;
}

}  // extern "C"

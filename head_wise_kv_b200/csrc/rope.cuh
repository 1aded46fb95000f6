// Rotary positions: the plan that kernels get by value, and the rotation of
// one thread's 16 elements, shared by rope.cu and append_rope.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "duo_internal.cuh"

struct duo_rope {
    duo_rope_desc desc;      // pair_factors cleared (not kept)
    double angle[64];        // radians per position of each pair
    double magnitude;
    uint64_t turn[64];       // the same as a fraction of a turn, times 2^64
};

namespace duo {

// A pair's angle at position p is p * f.  As a fraction of a turn in 64-bit
// fixed point the product wraps modulo whole turns by itself and adds no
// rounding of its own.  The fraction comes from a double, f / 2 pi within
// 2^-54 turns (f <= 1; thetas from 1.5 to 10^6 measured within 2^-55), so the
// angle is off by at most 2^-54 |p| turns: below fp32's rounding of what is
// left of it (2^-27 turns) up to |p| = 2^27, and 2^-23 turns, 7.5e-7 radians,
// at 2^31.  An fp32 angle at position 2^17 would be off by 2^-7 radians.
struct RopeTable {
    uint64_t turn[64];
    float magnitude;
    int rot_units;           // units (16 elements) of a head that rotate
    int half;                // 1: pairs (i, i + rot / 2), 0: (2i, 2i + 1)
};

inline RopeTable rope_table(const duo_rope* r) {
    RopeTable t;
    for (int i = 0; i < 64; ++i) t.turn[i] = r->turn[i];
    t.magnitude = float(r->magnitude);
    t.rot_units = r->desc.rot_dim / 16;
    t.half = r->desc.layout == DUO_ROPE_HALF;
    return t;
}

#ifdef __CUDACC__

// One thread's part of a head ("unit" u of head_dim / 16): two vectors of 8
// elements at offsets e0 and e1.  A unit that rotates holds the 8 pairs
// 8u .. 8u + 7: with pairs (i, i + rot / 2) the vectors are the pairs' two
// halves, with (2i, 2i + 1) they are neighbours.  The others are neighbours
// behind the first rot_dim elements and pass through.
struct RopeUnit {
    int e0, e1;
    bool rotates;
};

__device__ __forceinline__ RopeUnit rope_unit(const RopeTable& t, int u) {
    RopeUnit r;
    r.rotates = u < t.rot_units;
    const bool split = r.rotates && t.half;
    r.e0 = split ? 8 * u : 16 * u;
    r.e1 = split ? 8 * (u + t.rot_units) : 16 * u + 8;
    return r;
}

// Cosine and sine, times the magnitude, of a pair at position p.  The nearest
// quarter turn is taken off in fixed point, so that what becomes fp32 is at
// most 1/8 of a turn: its rounding moves the angle by at most 2^-24 of itself,
// about the rounding of the sine.
__device__ __forceinline__ void rope_angle(const RopeTable& t, int pair, int p, float sign, float& c, float& s) {
    const uint64_t a = uint64_t(int64_t(p)) * t.turn[pair];
    const uint32_t quarter = uint32_t((a + (uint64_t(1) << 61)) >> 62);
    const int64_t rest = int64_t(a - (uint64_t(quarter) << 62));
    float sn, cs;
    sincospif(float(rest) * 1.0842021724855044e-19f, &sn, &cs);      // 2^-63: in half turns
    const float cq = quarter & 1 ? sn : cs, sq = quarter & 1 ? cs : sn;
    c = (((quarter + 1) & 2) ? -cq : cq) * t.magnitude;
    s = ((quarter & 2) ? -sq : sq) * t.magnitude * sign;
}

// The same of pairs 8u .. 8u + 7.
__device__ __forceinline__ void rope_angles(const RopeTable& t, int u, int p, float sign, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rope_angle(t, 8 * u + i, p, sign, c[i], s[i]);
}

// x[0..7] and x[8..15] are the unit's two vectors.
template <bool HALF>
__device__ __forceinline__ void rope_rotate(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int a = HALF ? i : 2 * i, b = HALF ? i + 8 : 2 * i + 1;
        const float x0 = x[a], x1 = x[b];
        x[a] = x0 * c[i] - x1 * s[i];
        x[b] = x1 * c[i] + x0 * s[i];
    }
}

// Eight elements of a type: loaded as they are (so that several heads' loads
// are in flight), widened to fp32 exactly, rounded to nearest when stored.
template <typename T>
struct Vec8 {
    uint4 v;
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = v; }
};
template <>
struct Vec8<float> {
    uint4 v, w;
    __device__ __forceinline__ void load(const float* p) {
        v = reinterpret_cast<const uint4*>(p)[0];
        w = reinterpret_cast<const uint4*>(p)[1];
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<uint4*>(p)[0] = v;
        reinterpret_cast<uint4*>(p)[1] = w;
    }
};

__device__ __forceinline__ void widen(const Vec8<__nv_bfloat16>& v, float* x) {
    const uint32_t w[4] = {v.v.x, v.v.y, v.v.z, v.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf2_to_f2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void widen(const Vec8<__half>& v, float* x) {
    const uint32_t w[4] = {v.v.x, v.v.y, v.v.z, v.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void widen(const Vec8<float>& v, float* x) {
    const uint32_t w[8] = {v.v.x, v.v.y, v.v.z, v.v.w, v.w.x, v.w.y, v.w.z, v.w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}

__device__ __forceinline__ void narrow(Vec8<__nv_bfloat16>& v, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    v.v = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void narrow(Vec8<__half>& v, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    v.v = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void narrow(Vec8<float>& v, const float* x) {
    v.v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    v.w = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
}

#endif

// -------------------------------------------------------------- launch params
struct RopeTensor {
    const void* in;
    void* out;
    int64_t is_b, is_h, is_t, os_b, os_h, os_t;   // strides in elements
    int rotate;
};

struct RopeParams {
    RopeTensor t[3];
    int first_head[4];       // heads of the tensors before; [3] = all heads
    int B, n;
    int heads_per_thread;
    const int32_t* positions;
    int per_token;
    const int32_t* n_new;    // may be null
    float sign;              // -1: the transposed rotation
    RopeTable table;
};

cudaError_t launch_rope(const RopeParams& p, int dtype, int head_dim, int num_sms, cudaStream_t s);

}  // namespace duo

// linear_epilogue.h -- what the fused linear operators do to an element on its
// way to memory, shared by the tile kernels and the kernels that finish a
// split or compute gradients.
#pragma once

#include "gemm_internal.h"
#include "linear_internal.h"

namespace tra {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kChunk = 16 / sizeof(T);     // elements of a 16-byte chunk

// ---- activations -------------------------------------------------------------
//
// In binary32, with the formulas of the definitions:
//   gelu       z Phi(z);  slope Phi(z) + z phi(z)
//   gelu_tanh  z s,  s = sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3)), the tanh form
//              rewritten with 1 + tanh(a) = 2 sigmoid(2a)
//   silu       z sigmoid(z);  slope s (1 + z (1 - s))

__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

constexpr float kGeluA = 1.5957691216057308f;              // 2 sqrt(2 / pi)
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;

// NaN stays NaN, as in max(z, 0) of the array libraries.
__device__ __forceinline__ float relu(float z) { return z < 0.0f ? 0.0f : z; }

template <int V>
__device__ __forceinline__ void activate(int act, const float (&z)[V], float (&y)[V]) {
    switch (act) {
        case TRA_ACT_RELU:
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = relu(z[e]);
            break;
        case TRA_ACT_GELU:
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = 0.5f * z[e] * (1.0f + erff(z[e] * 0.70710678f));
            break;
        case TRA_ACT_GELU_TANH:
#pragma unroll
            for (int e = 0; e < V; ++e)
                y[e] = z[e] * sigmoid(z[e] * (kGeluA + kGeluB * z[e] * z[e]));
            break;
        case TRA_ACT_SILU:
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = z[e] * sigmoid(z[e]);
            break;
        case TRA_ACT_SIGMOID:
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = sigmoid(z[e]);
            break;
        default:
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = z[e];
    }
}

// y = act(z) and d = act'(z).
template <int V>
__device__ __forceinline__ void activate_slope(int act, const float (&z)[V], float (&y)[V],
                                               float (&d)[V]) {
    switch (act) {
        case TRA_ACT_RELU:
#pragma unroll
            for (int e = 0; e < V; ++e) {
                y[e] = relu(z[e]);
                d[e] = z[e] > 0.0f ? 1.0f : 0.0f;
            }
            break;
        case TRA_ACT_GELU:
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float cdf = 0.5f * (1.0f + erff(z[e] * 0.70710678f));
                y[e] = z[e] * cdf;
                d[e] = cdf + z[e] * 0.39894228f * __expf(-0.5f * z[e] * z[e]);
            }
            break;
        case TRA_ACT_GELU_TANH:
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float s = sigmoid(z[e] * (kGeluA + kGeluB * z[e] * z[e]));
                y[e] = z[e] * s;
                d[e] = s + y[e] * (1.0f - s) * (kGeluA + 3.0f * kGeluB * z[e] * z[e]);
            }
            break;
        case TRA_ACT_SILU:
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float s = sigmoid(z[e]);
                y[e] = z[e] * s;
                d[e] = s + y[e] * (1.0f - s);
            }
            break;
        case TRA_ACT_SIGMOID:
#pragma unroll
            for (int e = 0; e < V; ++e) {
                y[e] = sigmoid(z[e]);
                d[e] = y[e] * (1.0f - y[e]);
            }
            break;
        default:
#pragma unroll
            for (int e = 0; e < V; ++e) {
                y[e] = z[e];
                d[e] = 1.0f;
            }
    }
}

// ---- rows of V consecutive elements --------------------------------------------

// V elements from p, `valid` of them inside (the others read as zero);
// `vec`: p is 16-byte aligned.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T *p, int64_t valid, bool vec, float (&v)[V]) {
    constexpr int C = kChunk<T>;
    static_assert(V == 1 || V % C == 0, "one element or whole chunks");
    if (V > 1 && vec && valid >= V) {
#pragma unroll
        for (int c = 0; c < V / C; ++c) {
            T t[C];
            const u32x4 q = reinterpret_cast<const u32x4 *>(p)[c];
            __builtin_memcpy(t, &q, 16);
#pragma unroll
            for (int e = 0; e < C; ++e) v[c * C + e] = static_cast<float>(t[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = e < valid ? static_cast<float>(p[e]) : 0.0f;
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T *p, int64_t valid, bool vec, const float (&v)[V]) {
    constexpr int C = kChunk<T>;
    static_assert(V == 1 || V % C == 0, "one element or whole chunks");
    if (V > 1 && vec && valid >= V) {
#pragma unroll
        for (int c = 0; c < V / C; ++c) {
            T t[C];
#pragma unroll
            for (int e = 0; e < C; ++e) t[e] = static_cast<T>(v[c * C + e]);
            u32x4 q;
            __builtin_memcpy(&q, t, 16);
            reinterpret_cast<u32x4 *>(p)[c] = q;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < valid) p[e] = static_cast<T>(v[e]);
    }
}

// Finishes V (one, or a chunk of) elements of row m from column n on: z (and u)
// are the whole sums.  The one rounding to T is at the store; bias, activation
// and residual are binary32.
template <typename T, bool GATED, int V>
__device__ __forceinline__ void finish(const EpiArgs &e, int batch, int64_t m, int64_t n,
                                       float (&z)[V], float (&u)[V]) {
    const int64_t valid = e.N - n;
    float y[V];
    if constexpr (GATED) {
        if (e.Z != nullptr) {
            store_row<float, V>(e.Z + m * e.ldz + n, valid, e.vec_z, z);
            store_row<float, V>(e.Z + m * e.ldz + e.N + n, valid, e.vec_z, u);
        }
        activate(e.act, z, y);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] *= u[i];
    } else {
        if (e.bias != nullptr) {
            float b[V];
            load_row<T, V>(static_cast<const T *>(e.bias) + n, valid, e.vec_bias, b);
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] += b[i];
        }
        if (e.Z != nullptr) store_row<float, V>(e.Z + m * e.ldz + n, valid, e.vec_z, z);
        activate(e.act, z, y);
        if (e.R != nullptr) {
            float r[V];
            load_row<T, V>(static_cast<const T *>(e.R) + m * e.ldr + n, valid, e.vec_r, r);
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] += r[i];
        }
    }
    T *out = static_cast<T *>(batch == 0 ? e.Y[0] : e.Y[1]);
    store_row<T, V>(out + m * e.ldy + n, valid, e.vec_y, y);
}

}  // namespace
}  // namespace tra

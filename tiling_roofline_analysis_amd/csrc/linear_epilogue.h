// linear_epilogue.h -- what the fused linear operators do to an element on its
// way to memory, shared by the tile kernels and the kernels that finish a
// split or compute gradients.
#pragma once

#include <type_traits>

#include "gemm_internal.h"
#include "linear_internal.h"

namespace tra {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kChunk = 16 / sizeof(T);     // elements of a 16-byte chunk

// dZ is stored times a power of two, which the epilogue of its products undoes.
template <typename T>
constexpr bool kScaled = std::is_same_v<T, _Float16>;

// ---- activations -------------------------------------------------------------
//
// In binary32, with the formulas of the definitions:
//   gelu       z Phi(z);  slope Phi(z) + z phi(z).  For |z| < 1, Phi is 1/2 + z R(z^2);
//              beyond, Phi(-|z|) = 2^-Q(|z|).  R and Q are polynomials fitted by this
//              project to erf and to log2 Phi in 64 bits (least squares, reweighted
//              until the largest error, in units of what binary32 rounds gelu by, is
//              least; to |z| = 9, past which Q still rises).  gelu is off by at most
//              1.5e-7 of its value or 7e-8, as 0.5 z (1 + erf(z / sqrt 2)) in binary32
//              is, and keeps its size (to 4e-4) in the lower tail.  No branches: as
//              many steps as one rational approximation good to 1.5e-7 of Phi, which
//              is three to seven times as far off (2e-7 at z = -3)
//   gelu_tanh  z s,  s = sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3)), the tanh form
//              rewritten with 1 + tanh(a) = 2 sigmoid(2a)
//   silu       z sigmoid(z);  slope s (1 + z (1 - s))

__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

constexpr float kGeluA = 1.5957691216057308f;              // 2 sqrt(2 / pi)
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;

__device__ __forceinline__ float normal_cdf(float z) {
    const float a = fabsf(z), s = z * z;
    float r = 9.423413e-05f;
    r = r * s - 1.1693517e-03f;
    r = r * s + 9.967196e-03f;
    r = r * s - 6.6489585e-02f;
    r = r * s + 3.9894226e-01f;
    float q = 1.3285699e-06f;
    q = q * a - 5.052458e-05f;
    q = q * a + 8.353967e-04f;
    q = q * a - 8.090068e-03f;
    q = q * a + 5.292354e-02f;
    q = q * a + 4.5995072e-01f;
    q = q * a + 1.1500984e+00f;
    q = q * a + 1.0003642e+00f;
    q = __builtin_amdgcn_exp2f(-q);
    // (values, not expressions, to choose from: of those the compiler makes a branch for
    // every element, 4096 x 4096 x 256 in binary32 85 -> 92 us)
    const float inner = z * r + 0.5f, upper = 1.0f - q, outer = z > 0.0f ? upper : q;
    return a < 1.0f ? inner : outer;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    // NaN stays NaN, as in max(z, 0) of the array libraries
    if constexpr (ACT == TRA_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (ACT == TRA_ACT_GELU) return z * normal_cdf(z);
    if constexpr (ACT == TRA_ACT_GELU_TANH) return z * sigmoid(z * (kGeluA + kGeluB * z * z));
    if constexpr (ACT == TRA_ACT_SILU) return z * sigmoid(z);
    if constexpr (ACT == TRA_ACT_SIGMOID) return sigmoid(z);
    return z;
}

// y = act(z); returns act'(z).
template <int ACT>
__device__ __forceinline__ float activate_slope(float z, float &y) {
    if constexpr (ACT == TRA_ACT_RELU) {
        y = activate<ACT>(z);
        return z > 0.0f ? 1.0f : 0.0f;
    }
    if constexpr (ACT == TRA_ACT_GELU) {
        const float cdf = normal_cdf(z);
        y = z * cdf;
        return cdf + z * 0.39894228f * __builtin_amdgcn_exp2f(z * z * -0.72134752f);
    }
    if constexpr (ACT == TRA_ACT_GELU_TANH) {
        const float s = sigmoid(z * (kGeluA + kGeluB * z * z));
        y = z * s;
        // s is 0 or 1 long before |z| = 1000; z^2 must not overflow against it
        return s + y * (1.0f - s) * (kGeluA + 3.0f * kGeluB * fminf(z * z, 1e6f));
    }
    if constexpr (ACT == TRA_ACT_SILU) {
        const float s = sigmoid(z);
        y = z * s;
        return s + y * (1.0f - s);
    }
    if constexpr (ACT == TRA_ACT_SIGMOID) {
        y = sigmoid(z);
        return y * (1.0f - y);
    }
    y = z;
    return 1.0f;
}

// f(std::integral_constant<int, act>{}): the activation is chosen once for many
// elements.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case TRA_ACT_RELU: f(std::integral_constant<int, TRA_ACT_RELU>{}); break;
        case TRA_ACT_GELU: f(std::integral_constant<int, TRA_ACT_GELU>{}); break;
        case TRA_ACT_GELU_TANH: f(std::integral_constant<int, TRA_ACT_GELU_TANH>{}); break;
        case TRA_ACT_SILU: f(std::integral_constant<int, TRA_ACT_SILU>{}); break;
        case TRA_ACT_SIGMOID: f(std::integral_constant<int, TRA_ACT_SIGMOID>{}); break;
        default: f(std::integral_constant<int, TRA_ACT_NONE>{});
    }
}

// ---- rows of V consecutive elements --------------------------------------------
//
// V is one element or whole 16-byte chunks.  Vector loads and stores take any
// alignment of whole elements (gfx950 global memory instructions do).

template <typename T, int V>
__device__ __forceinline__ void load_row(const T *p, float (&v)[V]) {
    constexpr int C = V == 1 ? 1 : kChunk<T>;
    static_assert(V % C == 0, "whole chunks");
#pragma unroll
    for (int c = 0; c < V / C; ++c) {
        T t[C];
        __builtin_memcpy(t, p + c * C, C * sizeof(T));
#pragma unroll
        for (int e = 0; e < C; ++e) v[c * C + e] = static_cast<float>(t[e]);
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T *p, const float (&v)[V]) {
    constexpr int C = V == 1 ? 1 : kChunk<T>;
    static_assert(V % C == 0, "whole chunks");
#pragma unroll
    for (int c = 0; c < V / C; ++c) {
        T t[C];
#pragma unroll
        for (int e = 0; e < C; ++e) t[e] = static_cast<T>(v[c * C + e]);
        __builtin_memcpy(p + c * C, t, C * sizeof(T));
    }
}

// The same for a row that ends after `valid` of the V elements (the others
// read as zero).
template <typename T, int V>
__device__ __forceinline__ void load_part(const T *p, int64_t valid, float (&v)[V]) {
    if (valid >= V) {
        load_row<T, V>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = e < valid ? static_cast<float>(p[e]) : 0.0f;
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_part(T *p, int64_t valid, const float (&v)[V]) {
    if (valid >= V) {
        store_row<T, V>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < valid) p[e] = static_cast<T>(v[e]);
    }
}

// Finishes V elements of row m from column n on, of which `valid` = N - n are
// inside: z (and u) are the whole sums.  The one rounding to T is at the store;
// bias, activation and residual are binary32.
template <typename T, bool GATED, int ACT, int V>
__device__ __forceinline__ void finish(const EpiArgs &e, int batch, int64_t m, int64_t n,
                                       float (&z)[V], float (&u)[V]) {
    const int64_t valid = e.N - n;
    if constexpr (kScaled<T> && !GATED) {
        const float undo = e.undo != nullptr ? *e.undo : 1.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] *= undo;
    }
    if (!GATED && e.bias != nullptr) {
        float b[V];
        load_part<T, V>(static_cast<const T *>(e.bias) + n, valid, b);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] += b[i];
    }
    if (e.Z != nullptr) {
        store_part<float, V>(e.Z + m * e.ldz + n, valid, z);
        if constexpr (GATED) store_part<float, V>(e.Z + m * e.ldz + e.N + n, valid, u);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = GATED ? activate<ACT>(z[i]) * u[i] : activate<ACT>(z[i]);
    if (!GATED && e.R != nullptr) {
        float r[V];
        load_part<T, V>(static_cast<const T *>(e.R) + m * e.ldr + n, valid, r);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] += r[i];
    }
    T *out = static_cast<T *>(batch == 0 ? e.Y[0] : e.Y[1]);
    store_part<T, V>(out + m * e.ldy + n, valid, z);
}

}  // namespace
}  // namespace tra

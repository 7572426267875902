// norm.hip -- the norms around a block with its gate and the residual stream's
// scale, forward and backward (tra_norm, tra_norm_backward in include/tra_gemm.h).
// Errors come back as status codes; nothing throws across the ABI and nothing is
// allocated: scratch is the caller's workspace.
//
// Memory bounds all of it: a row is read once and kept in registers, E elements a
// lane, while its sums are taken (one for the mean of squares; for a layer norm the mean
// first, then the squares about it, so that a large mean costs no digits).  Rows too
// wide for that are read again for each sum, from L2.
#include "tra_gemm.h"

#include <algorithm>
#include <type_traits>

#include "linear_epilogue.h"
#include "operator_args.h"

namespace tra {
namespace {

struct NormArgs {
    int norm, post;
    int64_t M, D, per_group;           // rows that share a row of the vectors
    float scale, eps, inv_d;
    const void *X;
    int64_t ldx;
    const void *H;
    int64_t ldh;
    const void *weight, *bias, *gate, *post_weight, *post_bias;
    int64_t ld_weight, ld_bias, ld_gate, ld_post_weight, ld_post_bias;
    void *R;
    int64_t ldr;
    void *Y;
    int64_t ldy;
};

// The vectors' gradients, in the order of the sums.
enum { kWeight = 0, kBias = 1, kGate = 2, kPostWeight = 3, kPostBias = 4, kVectors = 5 };

struct NormGradArgs {
    NormArgs f;                        // R, Y: not used
    const void *dR;
    int64_t lddr;
    const void *dY;
    int64_t lddy;
    void *dX;
    int64_t lddx;
    void *dH;
    int64_t lddh;
    // Sums of one chunk of rows: chunk c of sum v at partial[v] + c * D; or null.
    float *partial[kVectors];
    int64_t chunks_per_group, rows_per_chunk;
    float *stats;                      // kStats floats a row, where sums are a kernel of their own
};

constexpr int kStats = 8;              // mean and 1 / deviation of H and R, means of g and g n

// ---- sums over a row ------------------------------------------------------------------

// Every lane's sum of its group of LANES lanes of the wave.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    static_assert(LANES == 16 || LANES == 64, "a quarter of a wave, or all of it");
#define TRA_DPP_ADD(ctrl) \
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ctrl, 0xf, 0xf, true))
    TRA_DPP_ADD(0xb1);     // lane ^ 1
    TRA_DPP_ADD(0x4e);     // lane ^ 2
    TRA_DPP_ADD(0x141);    // mirrored in its 8
    TRA_DPP_ADD(0x140);    // mirrored in its 16
#undef TRA_DPP_ADD
    if constexpr (LANES == 64) {
        typedef uint32_t pair __attribute__((ext_vector_type(2)));
        pair t = __builtin_bit_cast(pair, __builtin_amdgcn_permlane16_swap(
                                              __float_as_uint(v), __float_as_uint(v), false, false));
        v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
        t = __builtin_bit_cast(pair, __builtin_amdgcn_permlane32_swap(
                                         __float_as_uint(v), __float_as_uint(v), false, false));
        v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
    }
    return v;
}

// Sums over the LANES lanes of a row, the same in each.  Rows of several waves meet in
// LDS, in one of two places in turn: a wave that writes a place again has passed the
// barrier of the sum between, behind which nobody reads the sum before it.
template <int LANES, int BLOCK>
struct RowSum {
    static constexpr int WAVES = LANES / 64;     // of a row
    float *lds;                                  // 2 * (BLOCK / 64) pairs, 16-byte aligned
    int turn = 0;

    // N sums at once.
    template <int N>
    __device__ __forceinline__ void all(float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lanes_sum<LANES < 64 ? LANES : 64>(v[i]);
        if constexpr (WAVES > 1) {
            float *place = lds + turn * (BLOCK / 64) * 2;
            turn ^= 1;
            const int wave = static_cast<int>(threadIdx.x >> 6);
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) place[wave * N + i] = v[i];
            }
            __syncthreads();
            const float *row = place + wave / WAVES * WAVES * N;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += row[w * N + i];
        }
    }
    __device__ __forceinline__ void operator()(float &a, float &b) {
        float v[2] = {a, b};
        all(v);
        a = v[0];
        b = v[1];
    }
    __device__ __forceinline__ float operator()(float a) {
        float v[1] = {a};
        all(v);
        return v[0];
    }
};

// ---- a lane's part of a row ---------------------------------------------------------------

// Chunk c of a lane: V elements from (c * LANES + lane) * V on, zeros past the row's end.
// RAGGED: the row may end inside a chunk.  It has V elements or more, so every load is of V
// elements inside the row: a chunk past the end is read where it ends with the row and
// moved into place afterwards.  (With a path of its own for such a chunk the compiler waits
// for each load where the paths meet: the four rows that the backward pass reads came one
// after the other, 5.5 us a row of 4096 instead of 4.8.)
template <typename T, int LANES, int E, bool RAGGED>
struct LanePart {
    static constexpr int V = kChunk<T>;
    u32x4 chunk[E / V];

    __device__ __forceinline__ void load(const void *row, int lane, int D) {
#pragma unroll
        for (int c = 0; c < E / V; ++c) {
            const int at = (c * LANES + lane) * V;
            const T *p = static_cast<const T *>(row);
            if constexpr (RAGGED) {
                __builtin_memcpy(&chunk[c], p + (at < D - V ? at : D - V), 16);
            } else {
                chunk[c] = u32x4{};
                if (at < D) __builtin_memcpy(&chunk[c], p + at, 16);
            }
        }
    }
    __device__ __forceinline__ void get(int lane, int D, float (&v)[E]) {
        if (RAGGED && D < LANES * E) {
#pragma unroll
            for (int c = 0; c < E / V; ++c) {
                const int over = (c * LANES + lane + 1) * V - D;
                chunk[c] = drop_elements<T>(chunk[c], over < 0 ? 0 : over < V ? over : V);
            }
        }
#pragma unroll
        for (int c = 0; c < E / V; ++c) {
            T t[V];
            __builtin_memcpy(t, &chunk[c], 16);
#pragma unroll
            for (int e = 0; e < V; ++e) v[c * V + e] = static_cast<float>(t[e]);
        }
    }
};

template <typename T, int V, int LANES, int E>
__device__ __forceinline__ void store_lane(void *row, int lane, int64_t D, const float (&v)[E]) {
#pragma unroll
    for (int c = 0; c < E / V; ++c) {
        const int64_t at = (static_cast<int64_t>(c) * LANES + lane) * V;
        float t[V];
#pragma unroll
        for (int e = 0; e < V; ++e) t[e] = v[c * V + e];
        store_part<T, V>(static_cast<T *>(row) + at, D - at, t);
    }
}

// v - mean inside the row, 0 past its end.
template <int V, int LANES, int E>
__device__ __forceinline__ void subtract_mean(float (&v)[E], float mean, int lane, int64_t D) {
#pragma unroll
    for (int c = 0; c < E / V; ++c) {
        const int64_t left = D - (static_cast<int64_t>(c) * LANES + lane) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) v[c * V + e] = e < left ? v[c * V + e] - mean : 0.0f;
    }
}

__device__ __forceinline__ float inverse_deviation(float mean_square, float eps) {
    return 1.0f / sqrtf(mean_square + eps);
}

// v becomes (v - mean) / deviation; returns 1 / deviation.
template <int V, int LANES, int E, typename Sum>
__device__ __forceinline__ float normalize(float (&v)[E], int kind, const NormArgs &p, int lane,
                                           Sum &sum, float &mean) {
    mean = 0.0f;
    if (kind == TRA_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += v[e];
        mean = sum(s) * p.inv_d;
        subtract_mean<V, LANES>(v, mean, lane, p.D);
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += v[e] * v[e];
    const float inverse = inverse_deviation(sum(s) * p.inv_d, p.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= inverse;
    return inverse;
}
template <int V, int LANES, int E, typename Sum>
__device__ __forceinline__ float normalize(float (&v)[E], int kind, const NormArgs &p, int lane,
                                           Sum &sum) {
    float mean;
    return normalize<V, LANES>(v, kind, p, lane, sum, mean);
}

// Group `group`'s row of a vector.
template <typename P>
__device__ __forceinline__ const P *vector_row(const void *v, int64_t ld, int64_t group) {
    return static_cast<const P *>(v) + group * ld;
}

// A lane's part of a vector (of its own element type P, the rows' being T).  It is waited
// for where it is loaded, which is where it is used.  Not RAGGED: no row ends inside a chunk
// (8192 x 4096 bf16, norm: 25.3 us, 26.5 with a way for that).
template <typename T, typename P, int LANES, int E, bool RAGGED = true>
__device__ __forceinline__ void vector_lane(const void *vec, int64_t ld, int64_t group, int lane,
                                            int D, float (&v)[E]) {
    constexpr int V = kChunk<T>;
    const P *row = vector_row<P>(vec, ld, group);
#pragma unroll
    for (int c = 0; c < E / V; ++c) {
        const int at = (c * LANES + lane) * V;
        float t[V] = {};
        if constexpr (RAGGED) {
            load_part<P, V>(row + at, D - at, t);
        } else {
            if (at < D) load_row<P, V>(row + at, t);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) v[c * V + e] = t[e];
    }
}

template <int LANES>
constexpr int kBlock = LANES < 256 ? 256 : LANES;

// ---- forward ------------------------------------------------------------------------------

// What hides the memory's latency is the number of waves: 8 a SIMD, where the registers allow it.
// RAGGED takes 106 SGPRs, which leave 7: one workgroup of 1024 lanes a CU, not two.
// 8192 x 4096 bf16, add_norm with one weight: 48 us in a row of calls, 52 with the inputs from
// memory (5.1 TB/s); 1000 x 5461 f32, layer, with a gate: 26 and 30 (2.9 TB/s).
template <typename T, typename P, int LANES, int E, bool RAGGED>
__global__ __launch_bounds__(kBlock<LANES>, RAGGED || E > 8 ? 4 : LANES < 256 ? 7 : 8)
void norm_forward(const NormArgs p) {
    constexpr int V = kChunk<T>, BLOCK = kBlock<LANES>, ROWS = BLOCK / LANES;
    __shared__ __align__(16) float lds[4 * (BLOCK / 64)];
    lds_poison(lds, 4 * (BLOCK / 64));
    RowSum<LANES, BLOCK> sum{lds};
    const int lane = static_cast<int>(threadIdx.x) % LANES, D = static_cast<int>(p.D);
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS; first < p.M; first += step) {
        const int64_t own = first + static_cast<int>(threadIdx.x) / LANES;
        const bool inside = own < p.M;          // (a row past the last takes part, unseen)
        const int64_t m = inside ? own : p.M - 1;
        const int64_t group = m / p.per_group;
        LanePart<T, LANES, E, RAGGED> px, ph;
        px.load(static_cast<const T *>(p.X) + m * p.ldx, lane, D);
        if (p.H != nullptr) ph.load(static_cast<const T *>(p.H) + m * p.ldh, lane, D);
        auto times = [&](float (&v)[E], const void *vec, int64_t ld) __attribute__((always_inline)) {
            if (vec == nullptr) return;
            float t[E];
            vector_lane<T, P, LANES, E, RAGGED>(vec, ld, group, lane, D, t);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= t[e];
        };
        auto plus = [&](float (&v)[E], const void *vec, int64_t ld) __attribute__((always_inline)) {
            if (vec == nullptr) return;
            float t[E];
            vector_lane<T, P, LANES, E, RAGGED>(vec, ld, group, lane, D, t);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] += t[e];
        };
        float x[E];
        px.get(lane, D, x);
        if (p.H != nullptr) {
            float h[E];
            ph.get(lane, D, h);
            if (p.post != TRA_NORM_NONE) {
                normalize<V, LANES>(h, p.post, p, lane, sum);
                times(h, p.post_weight, p.ld_post_weight);
                plus(h, p.post_bias, p.ld_post_bias);
            }
            times(h, p.gate, p.ld_gate);
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = p.scale * x[e] + h[e];
            if (p.R != nullptr && inside)
                store_lane<T, V, LANES>(static_cast<T *>(p.R) + m * p.ldr, lane, D, x);
        }
        if (p.norm != TRA_NORM_NONE) {
            normalize<V, LANES>(x, p.norm, p, lane, sum);
            times(x, p.weight, p.ld_weight);
            plus(x, p.bias, p.ld_bias);
            if (inside) store_lane<T, V, LANES>(static_cast<T *>(p.Y) + m * p.ldy, lane, D, x);
        }
    }
}

// ---- wide rows --------------------------------------------------------------------------------
//
// A workgroup of 1024 lanes a row; each chunk of the row is worked out again from
// memory for every sum over it.

constexpr int kWideLanes = 1024;

// f(chunk) for each chunk of this lane's part of a row.
template <int V, typename F>
__device__ __forceinline__ void chunks_of(int64_t D, F f) {
    for (int64_t at = static_cast<int64_t>(threadIdx.x) * V; at < D; at += kWideLanes * V) f(at);
}

template <int V>
__device__ __forceinline__ void fill(float (&v)[V], float x) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = x;
}

// The vector's chunk, or `none`.
template <typename P, int V>
__device__ __forceinline__ void vector_chunk(const void *v, int64_t ld, int64_t group, int64_t at,
                                             int64_t D, float none, float (&t)[V]) {
    if (v == nullptr)
        fill<V>(t, none);
    else
        load_part<P, V>(vector_row<P>(v, ld, group) + at, D - at, t);
}

// Mean and 1 / deviation of what get(at, v) gives chunk by chunk.
template <int V, typename Get, typename Sum>
__device__ __forceinline__ void wide_stats(int kind, const NormArgs &p, Get get, Sum &sum,
                                           float &mean, float &inverse) {
    mean = 0.0f;
    float v[V], s = 0.0f;
    if (kind == TRA_NORM_LAYER) {
        chunks_of<V>(p.D, [&](int64_t at) {
            get(at, v);
#pragma unroll
            for (int e = 0; e < V; ++e) s += at + e < p.D ? v[e] : 0.0f;
        });
        mean = sum(s) * p.inv_d;
        s = 0.0f;
    }
    chunks_of<V>(p.D, [&](int64_t at) {
        get(at, v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = v[e] - mean;
            s += at + e < p.D ? d * d : 0.0f;
        }
    });
    inverse = inverse_deviation(sum(s) * p.inv_d, p.eps);
}

// Chunks of row m of H, of N_post(H) from its statistics, and of R.
template <typename T, typename P>
struct WideRow {
    static constexpr int V = kChunk<T>;
    const NormArgs &p;
    int64_t m, group;
    float mean_h = 0.0f, inv_h = 1.0f;

    __device__ __forceinline__ void h(int64_t at, float (&v)[V]) const {
        load_part<T, V>(static_cast<const T *>(p.H) + m * p.ldh + at, p.D - at, v);
    }
    // n: (h - mean) / deviation (h itself without a norm); behind: N_post(h)
    __device__ __forceinline__ void behind(int64_t at, float (&n)[V], float (&b)[V]) const {
        h(at, n);
#pragma unroll
        for (int e = 0; e < V; ++e) b[e] = n[e];
        if (p.post == TRA_NORM_NONE) return;
        float w[V], c[V];
        vector_chunk<P, V>(p.post_weight, p.ld_post_weight, group, at, p.D, 1.0f, w);
        vector_chunk<P, V>(p.post_bias, p.ld_post_bias, group, at, p.D, 0.0f, c);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            n[e] = (n[e] - mean_h) * inv_h;
            b[e] = n[e] * w[e] + c[e];
        }
    }
    __device__ __forceinline__ void r(int64_t at, float (&v)[V]) const {
        load_part<T, V>(static_cast<const T *>(p.X) + m * p.ldx + at, p.D - at, v);
        if (p.H == nullptr) return;
        float n[V], b[V], g[V];
        behind(at, n, b);
        vector_chunk<P, V>(p.gate, p.ld_gate, group, at, p.D, 1.0f, g);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = p.scale * v[e] + g[e] * b[e];
    }
};

template <typename T, typename P>
__global__ __launch_bounds__(kWideLanes) void norm_forward_wide(const NormArgs p) {
    constexpr int V = kChunk<T>;
    __shared__ __align__(16) float lds[4 * (kWideLanes / 64)];
    lds_poison(lds, 4 * (kWideLanes / 64));
    RowSum<kWideLanes, kWideLanes> sum{lds};
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        WideRow<T, P> row{p, m, m / p.per_group};
        if (p.H != nullptr && p.post != TRA_NORM_NONE)
            wide_stats<V>(p.post, p, [&](int64_t at, float (&v)[V]) { row.h(at, v); }, sum,
                          row.mean_h, row.inv_h);
        float mean = 0.0f, inverse = 1.0f;
        if (p.norm != TRA_NORM_NONE)
            wide_stats<V>(p.norm, p, [&](int64_t at, float (&v)[V]) { row.r(at, v); }, sum, mean,
                          inverse);
        // (R may be X: a lane reads its chunk for the last time before it writes it)
        chunks_of<V>(p.D, [&](int64_t at) {
            float v[V], w[V], b[V];
            row.r(at, v);
            if (p.R != nullptr)
                store_part<T, V>(static_cast<T *>(p.R) + m * p.ldr + at, p.D - at, v);
            if (p.norm == TRA_NORM_NONE) return;
            vector_chunk<P, V>(p.weight, p.ld_weight, row.group, at, p.D, 1.0f, w);
            vector_chunk<P, V>(p.bias, p.ld_bias, row.group, at, p.D, 0.0f, b);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = (v[e] - mean) * inverse * w[e] + b[e];
            store_part<T, V>(static_cast<T *>(p.Y) + m * p.ldy + at, p.D - at, v);
        });
    }
}

// ---- backward, rows in registers -----------------------------------------------------------------

// v: a row; g: the gradient of its norm's normalized row n.  v becomes n, and g the
// gradient of v, both 0 past the row's end.  The sums that depend on v only through its
// deviation are taken along with the one for that.
struct RowStats {
    float mean = 0.0f, inverse = 1.0f;     // of v
    float along = 0.0f, mean_g = 0.0f;     // means of g n and g
};
template <int V, int LANES, int E, typename Sum>
__device__ __forceinline__ RowStats normalize_both(float (&v)[E], float (&g)[E], int kind,
                                                   const NormArgs &p, int lane, Sum &sum) {
    RowStats s;
    if (kind == TRA_NORM_LAYER) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            a += v[e];
            b += g[e];
        }
        sum(a, b);
        s.mean = a * p.inv_d;
        s.mean_g = b * p.inv_d;
        subtract_mean<V, LANES>(v, s.mean, lane, p.D);
        subtract_mean<V, LANES>(g, s.mean_g, lane, p.D);
    }
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        a += v[e] * v[e];
        b += g[e] * v[e];
    }
    sum(a, b);
    s.inverse = inverse_deviation(a * p.inv_d, p.eps);
    s.along = b * s.inverse * p.inv_d;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        v[e] *= s.inverse;
        g[e] = s.inverse * (g[e] - v[e] * s.along);
    }
    return s;
}

// g: the gradient of a norm's normalized row n; becomes that of the row before it (0
// past the row's end, as it was).
template <int V, int LANES, int E, typename Sum>
__device__ __forceinline__ void normalize_gradient(float (&g)[E], const float (&n)[E],
                                                   float inverse, int kind, const NormArgs &p,
                                                   int lane, Sum &sum) {
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        a += g[e] * n[e];
        b += g[e];
    }
    sum(a, b);
    a *= p.inv_d;
    if (kind == TRA_NORM_LAYER) subtract_mean<V, LANES>(g, b * p.inv_d, lane, p.D);
#pragma unroll
    for (int e = 0; e < E; ++e) g[e] = inverse * (g[e] - n[e] * a);
}

// A workgroup takes a chunk of rows of one group, ROWS at a time, and keeps the sums of
// the vectors' gradients in registers until its end.  There are as many chunks as
// workgroups run at once, one or two a CU, since each costs a row of sums in memory; but a
// chunk for each group at least, where there are more of those.
// 8192 x 4096 bf16, norms before and behind the block and a gate: 88 us (4.6 TB/s); 1000 x 5461
// f32, layer, with biases: 38 (3.5 TB/s).
// POST: there is a norm of H.
// BIAS: gradients of biases are asked for.
constexpr int kBackwardBlock = 512;
// Workgroups a CU that the VGPRs leave room for.
constexpr int backward_per_cu(int64_t bytes, int64_t D, bool bias) {
    return bytes == 2 && D <= 4096 && !bias ? 2 : 1;
}

// Lanes of a row, and the rows that a workgroup takes at once: a chunk is of whole rounds of
// those, since a round takes its time however many of its rows are there (4096 x 128 bf16 in
// 4096 chunks of one row instead of 128 of 32: 30 us instead of 5; 1000 x 128 with the vectors'
// gradients in 500 chunks of two 16 instead of 13, and 16 times the workspace).
constexpr int backward_lanes(int64_t D) {
    return D <= 128 ? 16 : D <= 512 ? 64 : D <= 2048 ? 256 : 512;
}
constexpr int64_t backward_rows(int64_t D) { return kBackwardBlock / backward_lanes(D); }

template <typename T, typename P, int LANES, int E, bool POST, bool BIAS>
__global__ __launch_bounds__(kBackwardBlock, (2 * backward_per_cu(sizeof(T), LANES * E, BIAS)))
void norm_backward(const NormGradArgs q) {
    constexpr int V = kChunk<T>, BLOCK = kBackwardBlock, ROWS = BLOCK / LANES;
    const NormArgs &p = q.f;
    __shared__ __align__(16) float lds[4 * (BLOCK / 64)];
    __shared__ float part[ROWS > 1 ? (ROWS - 1) * LANES * E : 1];
    __shared__ __align__(16) float vectors[POST ? 4 : 2][LANES * E];
    lds_poison(&vectors[0][0], (POST ? 4 : 2) * LANES * E);
    lds_poison(lds, 4 * (BLOCK / 64));
    lds_poison(part, ROWS > 1 ? (ROWS - 1) * LANES * E : 1);
    RowSum<LANES, BLOCK> sum{lds};
    const int lane = static_cast<int>(threadIdx.x) % LANES;
    const int sub = static_cast<int>(threadIdx.x) / LANES, D = static_cast<int>(p.D);
    const int64_t group = blockIdx.x / q.chunks_per_group;
    const int64_t chunk = blockIdx.x - group * q.chunks_per_group;
    const int64_t begin = group * p.per_group + chunk * q.rows_per_chunk;
    const int64_t stop = (group + 1) * p.per_group;
    const int64_t end = begin + q.rows_per_chunk < stop ? begin + q.rows_per_chunk : stop;
    constexpr int SUMS = POST ? BIAS ? kVectors : kPostWeight + 1 : kGate + 1;
    float total[SUMS][E] = {};

    // The group's vectors, in LDS: waiting for a load from memory would wait for the rows
    // loaded ahead, too.
    auto keep = [&](float (&to)[LANES * E], const void *vec, int64_t ld, float none)
                    __attribute__((always_inline)) {
        float t[E];
#pragma unroll
        for (int e = 0; e < E; ++e) t[e] = none;
        if (vec != nullptr) vector_lane<T, P, LANES>(vec, ld, group, lane, D, t);
#pragma unroll
        for (int e = 0; e < E; ++e) to[(e / V * LANES + lane) * V + e % V] = t[e];
    };
    auto kept = [&](const float (&from)[LANES * E], int e) __attribute__((always_inline)) {
        return from[(e / V * LANES + lane) * V + e % V];
    };
    if (sub == 0) {
        keep(vectors[0], p.weight, p.ld_weight, 1.0f);
        keep(vectors[1], p.gate, p.ld_gate, 1.0f);
        if constexpr (POST) {
            keep(vectors[2], p.post_weight, p.ld_post_weight, 1.0f);
            keep(vectors[3], p.post_bias, p.ld_post_bias, 0.0f);
        }
    }
    __syncthreads();

    for (int64_t first = begin; first < end; first += ROWS) {
        // (a row past the last takes part, unseen: the last again, left out of the totals)
        const bool inside = ROWS == 1 || first + sub < end;
        const int64_t m = inside ? first + sub : end - 1;
        auto counted = [&](float v) __attribute__((always_inline)) { return inside ? v : 0.0f; };
        LanePart<T, LANES, E, true> x, y, dy, dr;          // (y: H)
        x.load(static_cast<const T *>(p.X) + m * p.ldx, lane, D);
        if (p.H != nullptr) y.load(static_cast<const T *>(p.H) + m * p.ldh, lane, D);
        if (q.dY != nullptr) dy.load(static_cast<const T *>(q.dY) + m * q.lddy, lane, D);
        if (q.dR != nullptr) dr.load(static_cast<const T *>(q.dR) + m * q.lddr, lane, D);
        float r[E], h[E] = {}, inv_h = 1.0f;
        x.get(lane, D, r);
        if (p.H != nullptr) y.get(lane, D, h);
        // N_post(H), from H normalized
        auto behind = [&](int e) __attribute__((always_inline)) {
            return POST ? h[e] * kept(vectors[POST ? 2 : 0], e) + kept(vectors[POST ? 3 : 0], e)
                        : h[e];
        };
        if (p.H != nullptr) {
            if constexpr (POST) inv_h = normalize<V, LANES>(h, p.post, p, lane, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) r[e] = p.scale * r[e] + kept(vectors[1], e) * behind(e);
        }
        // G, the gradient of R
        float g[E] = {};
        if (q.dY != nullptr) {
            float d[E];
            dy.get(lane, D, d);
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = d[e] * kept(vectors[0], e);
            normalize_both<V, LANES>(r, g, p.norm, p, lane, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                total[kWeight][e] += counted(d[e] * r[e]);
                if constexpr (BIAS) total[kBias][e] += counted(d[e]);
            }
        }
        if (q.dR != nullptr) {
            float d[E];
            dr.get(lane, D, d);
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] += d[e];
        }
        if (q.dX != nullptr && inside) {
            const float scale = p.H != nullptr ? p.scale : 1.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) r[e] = scale * g[e];
            store_lane<T, V, LANES>(static_cast<T *>(q.dX) + m * q.lddx, lane, p.D, r);
        }
        if (p.H != nullptr) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                total[kGate][e] += counted(g[e] * behind(e));
                g[e] *= kept(vectors[1], e);
            }
            if constexpr (POST) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    total[kPostWeight][e] += counted(g[e] * h[e]);
                    if constexpr (BIAS) total[kPostBias][e] += counted(g[e]);
                    g[e] *= kept(vectors[2], e);
                }
                normalize_gradient<V, LANES>(g, h, inv_h, p.post, p, lane, sum);
            }
            if (q.dH != nullptr && inside)
                store_lane<T, V, LANES>(static_cast<T *>(q.dH) + m * q.lddh, lane, p.D, g);
        }
    }
    for (int k = 0; k < kVectors; ++k) {
        if (q.partial[k] == nullptr) continue;
        float t[E];
#pragma unroll
        for (int j = 0; j < SUMS; ++j)
            if (k == j) {
#pragma unroll
                for (int e = 0; e < E; ++e) t[e] = total[j][e];
            }
        if constexpr (ROWS > 1) {
            __syncthreads();
            if (sub > 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) part[((sub - 1) * E + e) * LANES + lane] = t[e];
            }
            __syncthreads();
            if (sub > 0) continue;
            for (int s = 1; s < ROWS; ++s)
#pragma unroll
                for (int e = 0; e < E; ++e) t[e] += part[((s - 1) * E + e) * LANES + lane];
        }
        float *out = q.partial[k] + static_cast<int64_t>(blockIdx.x) * p.D;
#pragma unroll
        for (int c = 0; c < E / V; ++c) {
            const int64_t at = (static_cast<int64_t>(c) * LANES + lane) * V;
            float s[V];
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] = t[c * V + e];
            store_part<float, V>(out + at, p.D - at, s);
        }
    }
}

// ---- backward, rows in registers, sums by themselves -----------------------------------
//
// Rows that leave no registers for sums of the vectors' gradients: 1024 lanes a row; the rows'
// statistics go to memory and norm_columns, which reads the rows again, takes the sums from
// them.  2048 x 16384 bf16 without a norm of H: 116 us (3.5 TB/s) and 87 (3.1 TB/s read); with
// the rows read again from L2 for each of their sums, as norm_backward_wide does, 193 and 92.

template <typename T, typename P, int E>
__global__ __launch_bounds__(1024) void norm_backward_rows(const NormGradArgs q) {
    constexpr int V = kChunk<T>, LANES = 1024;
    constexpr bool LATE = E * sizeof(T) > 32;      // dY and dR are loaded where they are used
    const NormArgs &p = q.f;
    __shared__ __align__(16) float lds[4 * (LANES / 64)];
    lds_poison(lds, 4 * (LANES / 64));
    RowSum<LANES, LANES> sum{lds};
    const int lane = static_cast<int>(threadIdx.x), D = static_cast<int>(p.D);
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        const int64_t group = m / p.per_group;
        LanePart<T, LANES, E, true> x, y, dy, dr;          // (y: H)
        x.load(static_cast<const T *>(p.X) + m * p.ldx, lane, D);
        if (p.H != nullptr) y.load(static_cast<const T *>(p.H) + m * p.ldh, lane, D);
        if (!LATE && q.dY != nullptr)
            dy.load(static_cast<const T *>(q.dY) + m * q.lddy, lane, D);
        if (!LATE && q.dR != nullptr)
            dr.load(static_cast<const T *>(q.dR) + m * q.lddr, lane, D);
        auto times = [&](float (&v)[E], const void *vec, int64_t ld) __attribute__((always_inline)) {
            if (vec == nullptr) return;
            float t[E];
            vector_lane<T, P, LANES>(vec, ld, group, lane, D, t);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= t[e];
        };
        float r[E], h[E], g[E], mean_h = 0.0f, inv_h = 1.0f;
        x.get(lane, D, r);
        if (p.H != nullptr) {
            y.get(lane, D, h);
            if (p.post != TRA_NORM_NONE)
                inv_h = normalize<V, LANES>(h, p.post, p, lane, sum, mean_h);
            float b[E];
#pragma unroll
            for (int e = 0; e < E; ++e) b[e] = h[e];
            if (p.post != TRA_NORM_NONE) {
                times(b, p.post_weight, p.ld_post_weight);
                if (p.post_bias != nullptr) {
                    float t[E];
                    vector_lane<T, P, LANES>(p.post_bias, p.ld_post_bias, group, lane, D, t);
#pragma unroll
                    for (int e = 0; e < E; ++e) b[e] += t[e];
                }
            }
            times(b, p.gate, p.ld_gate);
#pragma unroll
            for (int e = 0; e < E; ++e) r[e] = p.scale * r[e] + b[e];
        }
        RowStats s;
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = 0.0f;
        if (q.dY != nullptr) {
            if (LATE) dy.load(static_cast<const T *>(q.dY) + m * q.lddy, lane, D);
            dy.get(lane, D, g);
            times(g, p.weight, p.ld_weight);
            s = normalize_both<V, LANES>(r, g, p.norm, p, lane, sum);
        }
        if (q.stats != nullptr && threadIdx.x == 0) {
            const float all[kStats] = {mean_h,  inv_h,    s.mean, s.inverse,
                                       s.along, s.mean_g, 0.0f,   0.0f};
#pragma unroll
            for (int i = 0; i < kStats; ++i) q.stats[m * kStats + i] = all[i];
        }
        if (q.dR != nullptr) {
            if (LATE) dr.load(static_cast<const T *>(q.dR) + m * q.lddr, lane, D);
            dr.get(lane, D, r);
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] += r[e];
        }
        if (q.dX != nullptr) {
            const float scale = p.H != nullptr ? p.scale : 1.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) r[e] = scale * g[e];
            store_lane<T, V, LANES>(static_cast<T *>(q.dX) + m * q.lddx, lane, p.D, r);
        }
        if (q.dH != nullptr) {
            times(g, p.gate, p.ld_gate);
            if (p.post != TRA_NORM_NONE) {
                times(g, p.post_weight, p.ld_post_weight);
                normalize_gradient<V, LANES>(g, h, inv_h, p.post, p, lane, sum);
            }
            store_lane<T, V, LANES>(static_cast<T *>(q.dH) + m * q.lddh, lane, p.D, g);
        }
    }
}

// ---- backward, wide rows ------------------------------------------------------------------------

// What is taken from dY by the norm before the next block: G, chunk by chunk.
template <typename T, typename P>
struct WideGrad {
    static constexpr int V = kChunk<T>;
    const NormGradArgs &q;
    const WideRow<T, P> &row;
    float mean = 0.0f, inverse = 1.0f, a = 0.0f, b = 0.0f;

    // n: R normalized; g: dY * weight
    __device__ __forceinline__ void parts(int64_t at, float (&n)[V], float (&dy)[V],
                                          float (&g)[V]) const {
        const NormArgs &p = q.f;
        row.r(at, n);
        load_part<T, V>(static_cast<const T *>(q.dY) + row.m * q.lddy + at, p.D - at, dy);
        vector_chunk<P, V>(p.weight, p.ld_weight, row.group, at, p.D, 1.0f, g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            n[e] = (n[e] - mean) * inverse;
            g[e] *= dy[e];
        }
    }
    __device__ __forceinline__ void gradient(int64_t at, float (&n)[V], float (&dy)[V],
                                             float (&g)[V]) const {
        fill<V>(g, 0.0f);
        if (q.dY != nullptr) {
            parts(at, n, dy, g);
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = inverse * (g[e] - n[e] * a - b);
        }
        if (q.dR != nullptr) {
            float d[V];
            load_part<T, V>(static_cast<const T *>(q.dR) + row.m * q.lddr + at, q.f.D - at, d);
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] += d[e];
        }
    }
};

template <typename T, typename P>
__global__ __launch_bounds__(kWideLanes) void norm_backward_wide(const NormGradArgs q) {
    constexpr int V = kChunk<T>;
    const NormArgs &p = q.f;
    __shared__ __align__(16) float lds[4 * (kWideLanes / 64)];
    lds_poison(lds, 4 * (kWideLanes / 64));
    RowSum<kWideLanes, kWideLanes> sum{lds};
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        WideRow<T, P> row{p, m, m / p.per_group};
        if (p.H != nullptr && p.post != TRA_NORM_NONE)
            wide_stats<V>(p.post, p, [&](int64_t at, float (&v)[V]) { row.h(at, v); }, sum,
                          row.mean_h, row.inv_h);
        WideGrad<T, P> grad{q, row};
        float n[V], dy[V], g[V], w[V], x[V];
        if (q.dY != nullptr) {
            wide_stats<V>(p.norm, p, [&](int64_t at, float (&v)[V]) { row.r(at, v); }, sum,
                          grad.mean, grad.inverse);
            float a = 0.0f, b = 0.0f;
            chunks_of<V>(p.D, [&](int64_t at) {
                grad.parts(at, n, dy, g);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    a += at + e < p.D ? g[e] * n[e] : 0.0f;
                    b += at + e < p.D ? g[e] : 0.0f;
                }
            });
            sum(a, b);
            grad.a = a * p.inv_d;
            grad.b = p.norm == TRA_NORM_LAYER ? b * p.inv_d : 0.0f;
        }
        if (q.stats != nullptr && threadIdx.x == 0) {
            const float s[kStats] = {row.mean_h, row.inv_h, grad.mean, grad.inverse,
                                     grad.a,     grad.b,    0.0f,      0.0f};
#pragma unroll
            for (int i = 0; i < kStats; ++i) q.stats[m * kStats + i] = s[i];
        }
        // the gradient of H normalized: G * gate * post_weight
        auto behind = [&](int64_t at, float (&nh)[V], float (&d)[V]) {
            grad.gradient(at, n, dy, d);
            row.behind(at, nh, x);
            vector_chunk<P, V>(p.gate, p.ld_gate, row.group, at, p.D, 1.0f, w);
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] *= w[e];
            if (p.post == TRA_NORM_NONE) return;
            vector_chunk<P, V>(p.post_weight, p.ld_post_weight, row.group, at, p.D, 1.0f, w);
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] *= w[e];
        };
        float a = 0.0f, b = 0.0f, nh[V], d[V];
        if (q.dH != nullptr && p.post != TRA_NORM_NONE) {
            chunks_of<V>(p.D, [&](int64_t at) {
                behind(at, nh, d);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    a += at + e < p.D ? d[e] * nh[e] : 0.0f;
                    b += at + e < p.D ? d[e] : 0.0f;
                }
            });
            sum(a, b);
            a *= p.inv_d;
            b = p.post == TRA_NORM_LAYER ? b * p.inv_d : 0.0f;
        }
        chunks_of<V>(p.D, [&](int64_t at) {
            if (q.dX != nullptr) {
                grad.gradient(at, n, dy, g);
#pragma unroll
                for (int e = 0; e < V; ++e) g[e] *= p.H != nullptr ? p.scale : 1.0f;
                store_part<T, V>(static_cast<T *>(q.dX) + m * q.lddx + at, p.D - at, g);
            }
            if (q.dH != nullptr) {
                behind(at, nh, d);
                if (p.post != TRA_NORM_NONE) {
#pragma unroll
                    for (int e = 0; e < V; ++e) d[e] = row.inv_h * (d[e] - nh[e] * a - b);
                }
                store_part<T, V>(static_cast<T *>(q.dH) + m * q.lddh + at, p.D - at, d);
            }
        });
    }
}

// V elements from `at` on, zeros past the row's end; TINY: of rows shorter than a chunk of 16
// bytes.  (As LanePart: with a path of its own for the end each load is waited for by itself.)
template <typename T, int V, bool TINY>
__device__ __forceinline__ void load_columns(const T *row, int64_t at, int64_t D, float (&v)[V]) {
    if constexpr (TINY) {
        load_part<T, V>(row + at, D - at, v);
    } else {
        constexpr int W = kChunk<T>;
#pragma unroll
        for (int c = 0; c < V; c += W) {
            const int64_t over = at + c + W - D;
            u32x4 chunk;
            __builtin_memcpy(&chunk, row + (over > 0 ? D - W : at + c), 16);
            chunk = drop_elements<T>(chunk, over <= 0 ? 0 : over < W ? static_cast<int>(over) : W);
            T t[W];
            __builtin_memcpy(t, &chunk, 16);
#pragma unroll
            for (int e = 0; e < W; ++e) v[c + e] = static_cast<float>(t[e]);
        }
    }
}

// The vectors' gradients from the rows' statistics: 64 chunks of columns by one chunk of
// rows per workgroup, whose four waves take every fourth row.
template <typename T, typename P, bool TINY>
__global__ __launch_bounds__(256) void norm_columns(const NormGradArgs q) {
    constexpr int V = kChunk<T>;
    const NormArgs &p = q.f;
    __shared__ float part[3][64 * V];
    lds_poison(&part[0][0], 3 * 64 * V);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t blocks = ceil_div(p.D, 64 * V);
    const int64_t id = blockIdx.x / blocks, at = ((blockIdx.x - id * blocks) * 64 + lane) * V;
    const int64_t group = id / q.chunks_per_group;
    const int64_t begin =
        group * p.per_group + (id - group * q.chunks_per_group) * q.rows_per_chunk;
    const int64_t stop = (group + 1) * p.per_group;
    const int64_t end = begin + q.rows_per_chunk < stop ? begin + q.rows_per_chunk : stop;
    float total[kVectors][V] = {};
    if (at < p.D) {
        float weight[V], gate[V], post_weight[V], post_bias[V];
        auto vector = [&](float (&v)[V], const void *vec, int64_t ld, float none)
                          __attribute__((always_inline)) {
            vector_chunk<P, V>(vec, ld, group, at, p.D, none, v);
        };
        vector(weight, p.weight, p.ld_weight, 1.0f);
        vector(gate, p.gate, p.ld_gate, 1.0f);
        vector(post_weight, p.post_weight, p.ld_post_weight, 1.0f);
        vector(post_bias, p.post_bias, p.ld_post_bias, 0.0f);
        auto row = [&](const void *v, int64_t ld, int64_t m, float (&to)[V])
                       __attribute__((always_inline)) {
            load_columns<T, V, TINY>(static_cast<const T *>(v) + m * ld, at, p.D, to);
        };
        for (int64_t m = begin + wave; m < end; m += 4) {
            float n[V] = {}, h[V] = {}, dy[V] = {}, g[V] = {};
            if (q.dY != nullptr) {
                row(p.X, p.ldx, m, n);
                row(q.dY, q.lddy, m, dy);
            }
            if (p.H != nullptr) row(p.H, p.ldh, m, h);
            if (q.dR != nullptr) row(q.dR, q.lddr, m, g);
            const float *s = q.stats + m * kStats;
            const float mean_h = s[0], inv_h = s[1], mean = s[2], inverse = s[3], along = s[4],
                        mean_g = s[5];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                // (of a post of none: 0 and 1)
                const float nh = (h[e] - mean_h) * inv_h, b = nh * post_weight[e] + post_bias[e];
                const float r = p.H != nullptr ? p.scale * n[e] + gate[e] * b : n[e];
                const float nr = (r - mean) * inverse;
                if (q.dY != nullptr) {
                    g[e] += inverse * (dy[e] * weight[e] - nr * along - mean_g);
                    total[kWeight][e] += dy[e] * nr;
                    total[kBias][e] += dy[e];
                }
                const float gg = g[e] * gate[e];
                total[kGate][e] += g[e] * b;
                total[kPostWeight][e] += gg * nh;
                total[kPostBias][e] += gg;
            }
        }
    }
    for (int k = 0; k < kVectors; ++k) {
        if (q.partial[k] == nullptr) continue;
        float t[V];
#pragma unroll
        for (int j = 0; j < kVectors; ++j)
            if (k == j) {
#pragma unroll
                for (int e = 0; e < V; ++e) t[e] = total[j][e];
            }
        __syncthreads();
        if (wave > 0) {
#pragma unroll
            for (int e = 0; e < V; ++e) part[wave - 1][e * 64 + lane] = t[e];
        }
        __syncthreads();
        if (wave > 0 || at >= p.D) continue;
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int e = 0; e < V; ++e) t[e] += part[w][e * 64 + lane];
        store_part<float, V>(q.partial[k] + id * p.D + at, p.D - at, t);
    }
}

// Adds the chunks' sums in order: 32 columns of one gradient's row per workgroup, whose
// groups of lanes take every GROUPS-th chunk and are added in order.
struct NormJoinArgs {
    const float *partial[kVectors];
    void *out[kVectors];
    int64_t rows[kVectors];            // of the gradient: 1, or the groups
    int64_t D, chunks, chunks_per_group;
};

constexpr int kJoin = 32;

// The loads' latency bounds it: with many chunks there are more groups (512 chunks of three
// sums of 4096 take 6.9 us with 8, 6.4 with 32; 63 of two sums 4 us less with 8), and a lane's
// loads go eight at a time, the last of them at the last chunk again (one at a time for the rest,
// 63 chunks of three sums of 5461 took 9.0 us, so 6.6).  Many are the chunks of a group of rows:
// with a vector that several groups share, whose sum is over all chunks, beside vectors of
// their own, 32 groups of lanes are too many for those (backward pass of 4096 x 1024 bf16, 4 groups
// 28.7 us with 8, 26.8 with 32, but 16 groups 29.3 and 31.2, 256 40 and 87).
template <typename P, int GROUPS>
__global__ __launch_bounds__(kJoin * GROUPS) void norm_join(const NormJoinArgs p) {
    __shared__ float part[GROUPS][kJoin];
    lds_poison(&part[0][0], GROUPS * kJoin);
    const int j = threadIdx.x % kJoin, lanes = threadIdx.x / kJoin;
    const int64_t blocks = ceil_div(p.D, kJoin);
    const int k = blockIdx.y;
    if (p.out[k] == nullptr) return;
    const int64_t rows = p.rows[k], each = rows == 1 ? p.chunks : p.chunks_per_group;
    for (int64_t id = blockIdx.x; id < rows * blocks; id += gridDim.x) {
        const int64_t row = id / blocks, n = (id - row * blocks) * kJoin + j;
        const float *from = p.partial[k] + row * each * p.D + n;
        float sum = 0.0f;
        if (n < p.D) {
            for (int64_t c = lanes; c < each; c += 8 * GROUPS) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int64_t at = c + u * GROUPS;
                    v[u] = from[(at < each ? at : each - 1) * p.D];
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) sum = c + u * GROUPS < each ? sum + v[u] : sum;
            }
        }
        __syncthreads();
        part[lanes][j] = sum;
        __syncthreads();
        if (lanes == 0 && n < p.D) {
#pragma unroll
            for (int i = 1; i < GROUPS; ++i) sum += part[i][j];
            static_cast<P *>(p.out[k])[row * p.D + n] = static_cast<P>(sum);
        }
    }
}

// ---- launches ----------------------------------------------------------------------------------

constexpr int64_t kMaxBlocks = 1 << 20;      // workgroups that take rows in turn

// Whether rows of D elements of `bytes` bytes are kept in registers: not those longer than
// 1024 lanes' 16 elements (2048 x 16384 bf16 forward 64 us, read again for each sum 79), nor
// those shorter than a chunk of 16 bytes.
constexpr bool in_registers(int64_t D, int64_t bytes) { return D * bytes >= 16 && D <= 16384; }

template <typename T, typename P, int LANES, int E>
hipError_t launch_forward(const NormArgs &a, hipStream_t s) {
    const int64_t blocks = ceil_div(a.M, kBlock<LANES> / LANES);
    const dim3 grid(static_cast<unsigned>(std::min(blocks, kMaxBlocks)));
    if (a.D % kChunk<T> == 0)
        norm_forward<T, P, LANES, E, false><<<grid, kBlock<LANES>, 0, s>>>(a);
    else
        norm_forward<T, P, LANES, E, true><<<grid, kBlock<LANES>, 0, s>>>(a);
    return hipGetLastError();
}

// 8 elements a lane, and as few lanes as that takes.  With the next larger number of them
// add_norm takes, in us (forward; backward): 65536 x 128 bf16 33 instead of 13; 47 instead of
// 22, 16384 x 512 30, 13; 46, 21, 4096 x 2048 18, 13; 28, 22, 2048 x 4096 20, 13 (forward).
template <typename T, typename P>
hipError_t forward_of(const NormArgs &a, hipStream_t s) {
    if (in_registers(a.D, sizeof(T))) {
        if (a.D <= 128) return launch_forward<T, P, 16, 8>(a, s);
        if (a.D <= 512) return launch_forward<T, P, 64, 8>(a, s);
        if (a.D <= 2048) return launch_forward<T, P, 256, 8>(a, s);
        if (a.D <= 4096) return launch_forward<T, P, 512, 8>(a, s);
        if (a.D <= 8192) return launch_forward<T, P, 1024, 8>(a, s);
        return launch_forward<T, P, 1024, 16>(a, s);
    }
    norm_forward_wide<T, P><<<dim3(static_cast<unsigned>(std::min(a.M, kMaxBlocks))), kWideLanes,
                              0, s>>>(a);
    return hipGetLastError();
}

// Whether the backward pass has a kernel that keeps such rows and the sums of the vectors'
// gradients in registers: with a norm of H, rows past 4096 leave room for few sums.  (Of
// 4096 x 5120 without a norm of H: bf16 59 us, in two kernels 109, f32 99 and 166; with one: bf16
// 95 and 142.)
constexpr bool backward_fits(int64_t D, int64_t bytes, bool post, bool bias) {
    return in_registers(D, bytes) && D <= 8192 &&
           (D <= 4096 || !post || (bytes == 2 && !bias));
}

template <typename T, typename P, int LANES, int E = 8>
hipError_t launch_backward(const NormGradArgs &a, int64_t chunks, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(chunks));
    const bool post = a.f.post != TRA_NORM_NONE;
    const bool bias = a.partial[kBias] != nullptr || a.partial[kPostBias] != nullptr;
#define TRA_BACKWARD(POST, BIAS) \
    norm_backward<T, P, LANES, E, POST, BIAS><<<grid, kBackwardBlock, 0, s>>>(a)
    if (!post) {
        bias ? TRA_BACKWARD(false, true) : TRA_BACKWARD(false, false);
    } else if (!bias) {
        if constexpr (backward_fits(LANES * E, sizeof(T), true, false)) TRA_BACKWARD(true, false);
    } else {
        if constexpr (backward_fits(LANES * E, sizeof(T), true, true)) TRA_BACKWARD(true, true);
    }
#undef TRA_BACKWARD
    return hipGetLastError();
}

template <typename T, typename P>
hipError_t backward_of(const NormGradArgs &a, int64_t chunks, bool fits, bool sums, hipStream_t s) {
    const int64_t D = a.f.D;
    if (fits) {
        switch (backward_lanes(D)) {
            case 16: return launch_backward<T, P, 16>(a, chunks, s);
            case 64: return launch_backward<T, P, 64>(a, chunks, s);
            case 256: return launch_backward<T, P, 256>(a, chunks, s);
            default:
                if (D <= 4096) return launch_backward<T, P, 512>(a, chunks, s);
                return launch_backward<T, P, 512, 16>(a, chunks, s);
        }
    }
    const dim3 rows(static_cast<unsigned>(std::min(a.f.M, kMaxBlocks)));
    if (!in_registers(D, sizeof(T)))
        norm_backward_wide<T, P><<<rows, kWideLanes, 0, s>>>(a);
    else if (D <= 8192)
        norm_backward_rows<T, P, 8><<<rows, 1024, 0, s>>>(a);
    else
        norm_backward_rows<T, P, 16><<<rows, 1024, 0, s>>>(a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || !sums) return err;
    const int64_t blocks = ceil_div(D, 64 * kChunk<T>);
    const dim3 grid(static_cast<unsigned>(chunks * blocks));
    if (D < kChunk<T>)
        norm_columns<T, P, true><<<grid, 256, 0, s>>>(a);
    else
        norm_columns<T, P, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename P>
hipError_t launch_join(const NormJoinArgs &a, hipStream_t s) {
    int64_t rows = 1;
    for (int k = 0; k < kVectors; ++k)
        if (a.out[k] != nullptr) rows = std::max(rows, a.rows[k]);
    const dim3 grid(static_cast<unsigned>(std::min(rows * ceil_div(a.D, kJoin), kMaxBlocks)),
                    kVectors);
    if (a.chunks_per_group > 128)
        norm_join<P, 32><<<grid, kJoin * 32, 0, s>>>(a);
    else
        norm_join<P, 8><<<grid, kJoin * 8, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace tra

namespace {

using namespace tra::host;
using tra::ceil_div;
using tra::NormArgs;
using tra::NormGradArgs;

constexpr int64_t kMaxGroups = 65535;

bool valid_kind(int k) { return k >= TRA_NORM_NONE && k < TRA_NORM_KIND_COUNT; }

// A vector: 1 or `groups` rows of D.
View vector_view(const void *p, int64_t ld, int64_t groups, int64_t D, int64_t bytes) {
    return View{p, p == nullptr ? 0 : ld == 0 ? 1 : groups, D, ld == 0 ? D : ld, bytes};
}

// What both directions check: types, kinds, sizes.
template <typename A>
tra_status check_common(const A &a) {
    if (!valid_dtype(a.dtype) || !valid_kind(a.norm) || !valid_kind(a.post) ||
        (a.param_dtype != a.dtype && a.param_dtype != TRA_DTYPE_F32) || a.M < 0 || a.D < 0 ||
        a.groups < 1 || a.M % a.groups != 0 || !(a.eps >= 0.0f))
        return TRA_ERR_INVALID_ARG;
    // (an empty matrix may be at NULL)
    if (a.H == nullptr && a.M > 0 && a.D > 0 && (a.post != TRA_NORM_NONE || a.gate != nullptr))
        return TRA_ERR_INVALID_ARG;
    if (a.post == TRA_NORM_NONE && (a.post_weight != nullptr || a.post_bias != nullptr))
        return TRA_ERR_INVALID_ARG;
    if (a.norm == TRA_NORM_NONE && (a.weight != nullptr || a.bias != nullptr))
        return TRA_ERR_INVALID_ARG;
    if (a.M > kMaxSize || a.D > kMaxSize || a.groups > kMaxGroups) return TRA_ERR_UNSUPPORTED;
    return TRA_OK;
}

// The inputs that both directions read (`biases`: the forward pass reads them).
template <typename A>
bool inputs_of(const A &a, bool biases, View (&in)[7]) {
    const int64_t b = elem_bytes(a.dtype), pb = elem_bytes(a.param_dtype);
    in[0] = View{a.X, a.M, a.D, a.ldx, b};
    in[1] = View{a.H, a.H != nullptr ? a.M : 0, a.D, a.ldh, b};
    in[2] = vector_view(a.weight, a.ld_weight, a.groups, a.D, pb);
    in[3] = vector_view(a.gate, a.ld_gate, a.groups, a.D, pb);
    in[4] = vector_view(a.post_weight, a.ld_post_weight, a.groups, a.D, pb);
    in[5] = vector_view(a.post_bias, a.ld_post_bias, a.groups, a.D, pb);
    in[6] = vector_view(biases ? a.bias : nullptr, a.ld_bias, a.groups, a.D, pb);
    for (const View &v : in)
        if (!v.valid()) return false;
    return true;
}

template <typename A>
NormArgs device_args(const A &a) {
    NormArgs d{};
    d.norm = a.norm;
    d.post = a.post;
    d.M = a.M;
    d.D = a.D;
    d.per_group = a.M / a.groups;
    d.scale = a.scale;
    d.eps = a.eps;
    d.inv_d = static_cast<float>(1.0 / static_cast<double>(a.D));
    d.X = a.X;
    d.ldx = a.ldx;
    d.H = a.H;
    d.ldh = a.ldh;
    d.weight = a.weight;
    d.bias = a.bias;
    d.gate = a.gate;
    d.post_weight = a.post_weight;
    d.post_bias = a.post_bias;
    d.ld_weight = a.ld_weight;
    d.ld_bias = a.ld_bias;
    d.ld_gate = a.ld_gate;
    d.ld_post_weight = a.ld_post_weight;
    d.ld_post_bias = a.ld_post_bias;
    return d;
}

// f<element type, parameter type>()
template <typename F>
hipError_t by_type(int dtype, int param_dtype, F f) {
    const bool f32 = param_dtype == TRA_DTYPE_F32;
    switch (dtype) {
        case TRA_DTYPE_F32: return f(0.0f, 0.0f);
        case TRA_DTYPE_BF16:
            return f32 ? f(__bf16(0.0f), 0.0f) : f(__bf16(0.0f), __bf16(0.0f));
        default: return f32 ? f(_Float16(0.0f), 0.0f) : f(_Float16(0.0f), _Float16(0.0f));
    }
}

// ---- forward ----------------------------------------------------------------------

tra_status check_forward(const tra_norm_args *p) {
    if (p == nullptr) return TRA_ERR_INVALID_ARG;
    const tra_norm_args &a = *p;
    const tra_status st = check_common(a);
    if (st != TRA_OK) return st;
    if ((a.norm != TRA_NORM_NONE) != (a.Y != nullptr) || (a.H == nullptr && a.R != nullptr) ||
        (a.Y == nullptr && a.R == nullptr)) {
        if (a.M > 0 && a.D > 0) return TRA_ERR_INVALID_ARG;
    }
    if (a.M == 0 || a.D == 0) return TRA_OK;
    const int64_t b = elem_bytes(a.dtype);
    View in[7];
    if (!inputs_of(a, true, in)) return TRA_ERR_INVALID_ARG;
    const View R{a.R, a.R != nullptr ? a.M : 0, a.D, a.ldr, b};
    const View Y{a.Y, a.Y != nullptr ? a.M : 0, a.D, a.ldy, b};
    if (!R.valid() || !Y.valid() || share(R, Y)) return TRA_ERR_INVALID_ARG;
    for (const View &v : in) {
        // X in place: the lane that reads an element of X writes it, after its last read
        const bool in_place = &v == &in[0] && same(v, R);
        if (share(v, Y) || (share(v, R) && !in_place)) return TRA_ERR_INVALID_ARG;
    }
    return TRA_OK;
}

tra_status forward(const tra_norm_args *p, void *stream) {
    const tra_status st = check_forward(p);
    if (st != TRA_OK || p->M == 0 || p->D == 0) return st;
    NormArgs d = device_args(*p);
    d.R = p->R;
    d.ldr = p->ldr;
    d.Y = p->Y;
    d.ldy = p->ldy;
    return status_of(by_type(p->dtype, p->param_dtype, [&](auto t, auto w) {
        return tra::forward_of<decltype(t), decltype(w)>(d, static_cast<hipStream_t>(stream));
    }));
}

// ---- backward ----------------------------------------------------------------------

struct GradPlan {
    int64_t chunks_per_group, rows_per_chunk, chunks;
    int vectors;               // gradients of vectors asked for
    size_t partial_bytes;      // of one
    size_t stats_bytes;
    size_t total;
    bool fits;                 // rows and sums in registers; else the rows' statistics are kept
};

bool wants(const tra_norm_grad_args &a, int k) {
    const void *out[] = {a.dweight, a.dbias, a.dgate, a.dpost_weight, a.dpost_bias};
    return out[k] != nullptr;
}

// Rows of the gradient of vector k.
int64_t rows_of(const tra_norm_grad_args &a, int k) {
    const int64_t ld[] = {a.ld_weight, a.ld_bias, a.ld_gate, a.ld_post_weight, a.ld_post_bias};
    return ld[k] == 0 ? 1 : a.groups;
}

GradPlan plan_backward(const tra_norm_grad_args &a) {
    GradPlan g{};
    for (int k = 0; k < tra::kVectors; ++k) g.vectors += wants(a, k);
    const bool bias = wants(a, tra::kBias) || wants(a, tra::kPostBias);
    const int64_t bytes = elem_bytes(a.dtype);
    g.fits = tra::backward_fits(a.D, bytes, a.post != TRA_NORM_NONE, bias);
    const int64_t per_group = a.M / a.groups;
    // as many workgroups as run at once where their sums are kept, or 8 a CU of those that
    // take sums alone (2048 x 16384 bf16: 100 us and 9 for the join of 256 chunks, 87 and 5
    // of 64); without sums as many as there are rounds of rows, to 4096
    int64_t most = 4096;
    if (g.vectors > 0)
        most = g.fits ? 256 * tra::backward_per_cu(bytes, a.D, bias)
                      : std::max<int64_t>(1, 2048 / ceil_div(a.D, 1024 / bytes));
    const int64_t want = std::max<int64_t>(1, most / a.groups);
    g.rows_per_chunk = std::max<int64_t>(1, ceil_div(per_group, want));
    if (g.fits) {
        const int64_t rows = tra::backward_rows(a.D);
        g.rows_per_chunk = ceil_div(g.rows_per_chunk, rows) * rows;
    }
    g.chunks_per_group = std::max<int64_t>(1, ceil_div(per_group, g.rows_per_chunk));
    g.chunks = a.groups * g.chunks_per_group;
    if (g.vectors > 0) {
        g.partial_bytes =
            align_up(static_cast<size_t>(g.chunks) * static_cast<size_t>(a.D) * sizeof(float));
        if (!g.fits)
            g.stats_bytes = align_up(static_cast<size_t>(a.M) * tra::kStats * sizeof(float));
    }
    g.total = g.vectors * g.partial_bytes + g.stats_bytes;
    return g;
}

tra_status check_backward(const tra_norm_grad_args *p) {
    if (p == nullptr) return TRA_ERR_INVALID_ARG;
    const tra_norm_grad_args &a = *p;
    const tra_status st = check_common(a);
    if (st != TRA_OK) return st;
    if (a.D == 0) return TRA_OK;
    if (a.H == nullptr && a.M > 0 && (a.dR != nullptr || a.dH != nullptr))
        return TRA_ERR_INVALID_ARG;
    if (a.norm == TRA_NORM_NONE && a.dY != nullptr) return TRA_ERR_INVALID_ARG;
    if ((a.dweight != nullptr && a.weight == nullptr) || (a.dgate != nullptr && a.gate == nullptr) ||
        (a.dpost_weight != nullptr && a.post_weight == nullptr) ||
        (a.dpost_bias != nullptr && a.post == TRA_NORM_NONE) ||
        (a.dbias != nullptr && a.norm == TRA_NORM_NONE))
        return TRA_ERR_INVALID_ARG;
    const int64_t b = elem_bytes(a.dtype), pb = elem_bytes(a.param_dtype);
    View in[7];
    if (!inputs_of(a, false, in)) return TRA_ERR_INVALID_ARG;
    const View dR{a.dR, a.dR != nullptr ? a.M : 0, a.D, a.lddr, b};
    const View dY{a.dY, a.dY != nullptr ? a.M : 0, a.D, a.lddy, b};
    if (!dR.valid() || !dY.valid()) return TRA_ERR_INVALID_ARG;
    void *const vectors[] = {a.dweight, a.dbias, a.dgate, a.dpost_weight, a.dpost_bias};
    View out[7];
    out[0] = View{a.dX, a.dX != nullptr ? a.M : 0, a.D, a.lddx, b};
    out[1] = View{a.dH, a.dH != nullptr ? a.M : 0, a.D, a.lddh, b};
    for (int k = 0; k < tra::kVectors; ++k)
        out[2 + k] = View{vectors[k], vectors[k] != nullptr ? rows_of(a, k) : 0, a.D, a.D, pb};
    for (int i = 0; i < 7; ++i) {
        if (!out[i].valid() || share(out[i], dR) || share(out[i], dY)) return TRA_ERR_INVALID_ARG;
        for (const View &v : in)
            if (share(out[i], v)) return TRA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return TRA_ERR_INVALID_ARG;
    }
    const GradPlan g = plan_backward(a);
    if (g.chunks * ceil_div(a.D, 256) * 256 > tra::kMaxGridLanes) return TRA_ERR_UNSUPPORTED;
    return TRA_OK;
}

tra_status backward(const tra_norm_grad_args *p, void *stream_) {
    const tra_status st = check_backward(p);
    if (st != TRA_OK || p->D == 0) return st;
    const tra_norm_grad_args &a = *p;
    const GradPlan g = plan_backward(a);
    if (!workspace_ok(a.workspace, a.workspace_bytes, g.total)) return TRA_ERR_INVALID_ARG;
    const hipStream_t stream = static_cast<hipStream_t>(stream_);
    NormGradArgs d{};
    d.f = device_args(a);
    d.dR = a.dR;
    d.lddr = a.lddr;
    d.dY = a.dY;
    d.lddy = a.lddy;
    d.dX = a.dX;
    d.lddx = a.lddx;
    d.dH = a.dH;
    d.lddh = a.lddh;
    d.chunks_per_group = g.chunks_per_group;
    d.rows_per_chunk = g.rows_per_chunk;
    char *ws = static_cast<char *>(a.workspace);
    if (g.stats_bytes > 0) d.stats = reinterpret_cast<float *>(ws);
    ws += g.stats_bytes;
    void *const vectors[] = {a.dweight, a.dbias, a.dgate, a.dpost_weight, a.dpost_bias};
    tra::NormJoinArgs j{};
    j.D = a.D;
    j.chunks = a.M > 0 ? g.chunks : 0;
    j.chunks_per_group = a.M > 0 ? g.chunks_per_group : 0;
    for (int k = 0; k < tra::kVectors; ++k) {
        if (!wants(a, k)) continue;
        j.partial[k] = d.partial[k] = reinterpret_cast<float *>(ws);
        ws += g.partial_bytes;
        j.out[k] = vectors[k];
        j.rows[k] = rows_of(a, k);
    }
    hipError_t err = hipSuccess;
    if (a.M > 0 && (a.dX != nullptr || a.dH != nullptr || g.vectors > 0))
        err = by_type(a.dtype, a.param_dtype, [&](auto t, auto w) {
            return tra::backward_of<decltype(t), decltype(w)>(d, g.chunks, g.fits, g.vectors > 0,
                                                             stream);
        });
    if (err == hipSuccess && g.vectors > 0)
        err = a.param_dtype == TRA_DTYPE_F32    ? tra::launch_join<float>(j, stream)
              : a.param_dtype == TRA_DTYPE_BF16 ? tra::launch_join<__bf16>(j, stream)
                                                : tra::launch_join<_Float16>(j, stream);
    return status_of(err);
}

}  // namespace

extern "C" {

tra_status tra_norm(const tra_norm_args *args, void *stream) { return forward(args, stream); }

tra_status tra_norm_backward(const tra_norm_grad_args *args, void *stream) {
    return backward(args, stream);
}

tra_status tra_norm_backward_workspace_size(const tra_norm_grad_args *args, size_t *bytes) {
    const tra_status st = check_backward(args);
    if (st != TRA_OK || bytes == nullptr) return st != TRA_OK ? st : TRA_ERR_INVALID_ARG;
    *bytes = args->D == 0 ? 0 : plan_backward(*args).total;
    return TRA_OK;
}

}  // extern "C"

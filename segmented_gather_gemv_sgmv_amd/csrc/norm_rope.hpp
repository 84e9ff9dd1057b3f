// norm_rope.hpp -- norms of queries and keys for each head, with the rotation
// of their positions in the same pass, and their gradients.
//
// A head x of D elements with weights w becomes
//     r = 1 / sqrt(mean(x^2) + eps),   n = x r w,   y = m Rot(t) n,
// Rot as in rope.hpp (angles from float64, pairs of the first `rot` elements).
// The gradients, from dy:
//     dn = m Rot(-t) dy,   dw = sum over rows and heads of dn x r,
//     dx = r w dn - x r^3 mean(w dn x).
//
// Bound: HBM (forward x in and y out, backward x and dy in and dx out; about
// ten flops an element), at decode sizes the launch.  So a head stays in
// registers between its sum and its output: L lanes (a power of two) hold a
// head, K units each, and the sums over a head are DPP moves and lane swaps
// within a wave.  A workgroup takes several rows at once, so that the angles
// of all of them are computed by all of its threads (one row alone has 64
// angles for 256 threads) and heads fill whole passes.
//
// Sums, statistics and weights' gradients are float32; outputs are rounded
// once.  The weights' gradients are summed by threads over the rows and heads
// they visit, by workgroups through LDS, and over workgroups by a second
// kernel, always in the same order.
#pragma once

#include <type_traits>

#include "norm_plan.hpp"
#include "sgmv_device.hpp"

namespace sgmv {

struct NormRopeArgs {
    void* out[2];                       // y; backward: dx (NULL: not wanted)
    const void* in[2];                  // x
    const void* grad[2];                // backward: dy
    const void* weight[2];              // NULL: ones
    long long in_row[2], in_head[2];    // strides in elements; the last dim's is 1
    long long out_row[2], out_head[2];
    long long grad_row[2], grad_head[2];
    float* partial;                     // backward: [workgroup][2][D]
    int sums[2];                        // backward: the weights' gradients that are wanted
    const void* positions;
    int wide_positions;
    const double* freq;
    float mag, eps, inv_D;
    int rows, heads[2], D, rot;
    int rows_per_block, blocks;         // rows of a workgroup at a time; blocks of rows
    int heads_per_group, groups;        // forward: head groups of a block, one workgroup each
    int units, lanes;                   // per head
    int interleaved;
};

// Sum over the `lanes` (a power of two) neighbouring lanes that hold a head; every lane
// gets it.  Within 16 lanes by DPP: quads swapped, halves of 8 and of 16 mirrored.
__device__ __forceinline__ float head_sum(float v, int lanes) {
    auto dpp = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value,
                                                          0xf, 0xf, true));
    };
    if (lanes > 1) v += dpp(v, std::integral_constant<int, 0xB1>{});
    if (lanes > 2) v += dpp(v, std::integral_constant<int, 0x4E>{});
    if (lanes > 4) v += dpp(v, std::integral_constant<int, 0x141>{});
    if (lanes > 8) v += dpp(v, std::integral_constant<int, 0x140>{});
    if (lanes > 16) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if (lanes > 32) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    return v;
}

// A thread's units of a head.  Unit u is V elements of each half that turn against each
// other (half layout), V elements of V / 2 interleaved pairs (or one pair, two
// elements, when V is 1), or V elements that do not turn.  kVec: V elements are 16 bytes
// and every address is a multiple of that; V is 1 otherwise.
template <typename DT, bool kVec, int K>
struct HeadUnits {
    using T = typename DT::storage;
    static constexpr int V = kVec ? 16 / DT::kBytes : 1;
    using Piece = std::conditional_t<kVec, uint4, T>;
    int at[K], second[K];   // first element, distance of the second piece (0: none)
    int u[K];               // unit, -1: none
    bool turned[K];

    __device__ __forceinline__ void init(const NormRopeArgs& a, int lane) {
        const int half = a.rot / 2;
        const int n_turned = a.interleaved ? (kVec ? a.rot / V : half) : half / V;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = lane + k * a.lanes;
            u[k] = i < a.units ? i : -1;
            turned[k] = i < n_turned;
            at[k] = !turned[k] ? a.rot + (i - n_turned) * V : a.interleaved ? (kVec ? i * V : 2 * i) : i * V;
            second[k] = !turned[k] ? 0 : a.interleaved ? (kVec ? 0 : 1) : half;
        }
    }
    // Both pieces of every unit from a head's first element; absent ones are zeros.
    struct Raw {
        Piece x[K], y[K];
    };
    __device__ __forceinline__ void load(const T* p, Raw& r) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            r.x[k] = Piece{};
            r.y[k] = Piece{};
            if (u[k] < 0) continue;
            r.x[k] = *reinterpret_cast<const Piece*>(p + at[k]);
            if (second[k]) r.y[k] = *reinterpret_cast<const Piece*>(p + at[k] + second[k]);
        }
    }
    __device__ static __forceinline__ void unpack(const Piece& p, float* f) {
        if constexpr (kVec) DT::unpack(p, f);
        else f[0] = DT::load1(&p);
    }
    __device__ __forceinline__ void floats(const Raw& r, float (*f)[2 * V]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            unpack(r.x[k], f[k]);
            unpack(r.y[k], f[k] + V);
        }
    }
    __device__ __forceinline__ void store(T* p, float (*f)[2 * V]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (u[k] < 0) continue;
            if constexpr (kVec) {
                store16(p + at[k], DT::pack(f[k]));
                if (second[k]) store16(p + at[k] + second[k], DT::pack(f[k] + V));
            } else {
                p[at[k]] = DT::from_float(f[k][0]);
                if (second[k]) p[at[k] + second[k]] = DT::from_float(f[k][1]);
            }
        }
    }
    // Turns the units by the angles of their row (cosine and sine times the magnitude).
    __device__ __forceinline__ void turn(float (*f)[2 * V], const float* c, const float* s, bool pairs_inside,
                                         float sign) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!turned[k] || u[k] < 0) continue;
            if (kVec && pairs_inside) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float cc = c[u[k] * (V / 2) + i], ss = s[u[k] * (V / 2) + i] * sign;
                    const float x = f[k][2 * i], y = f[k][2 * i + 1];
                    f[k][2 * i] = x * cc - y * ss;
                    f[k][2 * i + 1] = y * cc + x * ss;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float cc = c[u[k] * V + i], ss = s[u[k] * V + i] * sign;
                    const float x = f[k][i], y = f[k][V + i];
                    f[k][i] = x * cc - y * ss;
                    f[k][V + i] = y * cc + x * ss;
                }
            }
        }
    }
};

// Cosines and sines (times the magnitude) of rows [row0, row0 + rows) into LDS.
__device__ __forceinline__ void norm_angles(const NormRopeArgs& a, int row0, int rows, float* s_cos,
                                            float* s_sin) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < rows * half; i += kNormThreads) {
        const int r = i / half, j = i - r * half;
        const double pos = a.wide_positions ? (double)((const long long*)a.positions)[row0 + r]
                                            : (double)((const int*)a.positions)[row0 + r];
        // fraction of a turn in [-1/2, 1/2], times 2: sincospi's argument
        const double t = pos * a.freq[j] * 0.15915494309189533577;
        float sn, cs;
        sincospif(2.f * (float)(t - rint(t)), &sn, &cs);
        s_cos[i] = cs * a.mag;
        s_sin[i] = sn * a.mag;
    }
}

template <typename DT, bool kVec, int K>
__global__ __launch_bounds__(kNormThreads) void norm_rope_kernel(NormRopeArgs a) {
    using Units = HeadUnits<DT, kVec, K>;
    using T = typename DT::storage;
    constexpr int V = Units::V;
    __shared__ float s_cos[kNormAngles], s_sin[kNormAngles];
    const int blk = (int)(blockIdx.x / (unsigned)a.groups);
    const int grp = (int)(blockIdx.x - (unsigned)blk * a.groups);
    const int row0 = blk * a.rows_per_block;
    const int rows = min(a.rows_per_block, a.rows - row0);
    const int h_lo = grp * a.heads_per_group;
    const int hn = min(a.heads_per_group, a.heads[0] + a.heads[1] - h_lo);
    const int lane = threadIdx.x & (a.lanes - 1), step = kNormThreads / a.lanes;
    const int items = rows * hn, half = a.rot / 2;
    Units un;
    un.init(a, lane);

    // Item it: row it / hn, head it % hn of the group.
    auto place = [&](int it, int& r, int& w, int& h) {
        r = it / hn;
        h = h_lo + it - r * hn;
        w = h >= a.heads[0];
        if (w) h -= a.heads[0];
    };
    typename Units::Raw raw;
    auto load = [&](int it) {
        int r, w, h;
        place(it, r, w, h);
        un.load((const T*)a.in[w] + (long long)(row0 + r) * a.in_row[w] + (long long)h * a.in_head[w], raw);
    };
    int it = threadIdx.x / a.lanes;
    if (it < items) load(it);
    norm_angles(a, row0, rows, s_cos, s_sin);
    __syncthreads();
    for (; it < items; it += step) {
        float f[K][2 * V];
        un.floats(raw, f);
        int r, w, h;
        place(it, r, w, h);
        if (it + step < items) load(it + step);  // the next head, behind this one's sums
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) ss += f[k][i] * f[k][i];
        const float rs = 1.f / sqrtf(head_sum(ss, a.lanes) * a.inv_D + a.eps);
        if (a.weight[w]) {
            typename Units::Raw wr;
            float wf[K][2 * V];
            un.load((const T*)a.weight[w], wr);
            un.floats(wr, wf);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) f[k][i] = f[k][i] * rs * wf[k][i];
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) f[k][i] *= rs;
        }
        un.turn(f, s_cos + r * half, s_sin + r * half, a.interleaved, 1.f);
        un.store((T*)a.out[w] + (long long)(row0 + r) * a.out_row[w] + (long long)h * a.out_head[w], f);
    }
}

// Gradients.  Workgroup b takes the blocks of rows b, b + gridDim.x, ...; its threads keep
// the sums of the weights' gradients over all of them.
template <typename DT, bool kVec, int K>
__global__ __launch_bounds__(kNormThreads) void norm_rope_grad_kernel(NormRopeArgs a) {
    using Units = HeadUnits<DT, kVec, K>;
    using T = typename DT::storage;
    constexpr int V = Units::V;
    __shared__ float s_cos[kNormAngles], s_sin[kNormAngles];
    __shared__ float s_sum[kNormThreads];
    const int lane = threadIdx.x & (a.lanes - 1), step = kNormThreads / a.lanes, half = a.rot / 2;
    const int slot = threadIdx.x / a.lanes;
    Units un;
    un.init(a, lane);
    float acc[2][K][2 * V] = {};
    for (int blk = blockIdx.x; blk < a.blocks; blk += gridDim.x) {
        const int row0 = blk * a.rows_per_block;
        const int rows = min(a.rows_per_block, a.rows - row0);
        __syncthreads();
        norm_angles(a, row0, rows, s_cos, s_sin);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int hn = a.heads[w], items = rows * hn;
            if (items == 0) continue;
            float wf[K][2 * V];
            if (a.weight[w]) {
                typename Units::Raw wr;
                un.load((const T*)a.weight[w], wr);
                un.floats(wr, wf);
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) wf[k][i] = 1.f;
            }
            typename Units::Raw rx, rg;
            auto load = [&](int it) {
                const int r = it / hn, h = it - r * hn;
                un.load((const T*)a.in[w] + (long long)(row0 + r) * a.in_row[w] + (long long)h * a.in_head[w], rx);
                un.load((const T*)a.grad[w] + (long long)(row0 + r) * a.grad_row[w] + (long long)h * a.grad_head[w], rg);
            };
            int it = slot;
            if (it < items) load(it);
            for (; it < items; it += step) {
                const int r = it / hn, h = it - r * hn;
                float x[K][2 * V], g[K][2 * V];
                un.floats(rx, x);
                un.floats(rg, g);
                if (it + step < items) load(it + step);
                un.turn(g, s_cos + r * half, s_sin + r * half, a.interleaved, -1.f);
                float ss = 0.f, dot = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) {
                        ss += x[k][i] * x[k][i];
                        dot += g[k][i] * wf[k][i] * x[k][i];
                    }
                ss = head_sum(ss, a.lanes);
                dot = head_sum(dot, a.lanes);
                const float rs = 1.f / sqrtf(ss * a.inv_D + a.eps);
                const float back = rs * rs * (dot * a.inv_D);
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) {
                        acc[w][k][i] += g[k][i] * (x[k][i] * rs);
                        g[k][i] = rs * (g[k][i] * wf[k][i] - x[k][i] * back);
                    }
                if (a.out[w])
                    un.store((T*)a.out[w] + (long long)(row0 + r) * a.out_row[w] + (long long)h * a.out_head[w], g);
            }
        }
    }
    // Over the workgroup's heads, element by element of a thread's units.
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (!a.sums[w]) continue;
        float* out = a.partial + ((long long)blockIdx.x * 2 + w) * a.D;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) {
                __syncthreads();
                s_sum[threadIdx.x] = acc[w][k][i];
                __syncthreads();
                if (slot == 0 && un.u[k] >= 0 && (i < V || un.second[k])) {
                    float t = 0.f;
                    for (int s = 0; s < step; ++s) t += s_sum[s * a.lanes + lane];
                    out[un.at[k] + (i < V ? i : un.second[k] + i - V)] = t;
                }
            }
    }
}

// The weights' gradients: sums of n partials per element, rounded once.  Workgroup (x, w) has
// 64 elements; thread (e, g) sums every 16th partial from g, then these are added in order.
template <typename DT>
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* partial, void* dwq, void* dwk, int n, int D) {
    using T = typename DT::storage;
    __shared__ float s[16][64];
    const int w = blockIdx.y, e = threadIdx.x & 63, g = threadIdx.x / 64;
    const int d = blockIdx.x * 64 + e;
    T* out = (T*)(w ? dwk : dwq);
    if (!out) return;
    float t = 0.f;
    if (d < D)
        for (int i = g; i < n; i += 16) t += partial[((long long)i * 2 + w) * D + d];
    s[g][e] = t;
    __syncthreads();
    if (g == 0 && d < D) {
        for (int i = 1; i < 16; ++i) t += s[i][e];
        out[d] = DT::from_float(t);
    }
}

}  // namespace sgmv

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
// ten flops an element), at decode sizes the launch.  Measured, heads of
// 128: 4096 rows of 32 + 8 in float16 17 us (a large copy of these 84 MB: 16), 8191 rows of 16 + 4 in
// bfloat16 18 us and their gradients 35 + 4 (126 MB: 24).
// So a head stays in
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
    float* partial;                     // backward: [workgroup][D]
    int split, grad_rows[2];            // backward: the queries' workgroups, rows of a block
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

// Two floats to two packed 16-bit values, nearest-even, bfloat16 by the packed conversion.
template <typename DT>
__device__ __forceinline__ uint32_t norm_pack2(float lo, float hi) {
    if constexpr (std::is_same<DT, BF16>::value) {
        typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
        const b2_t v = {(__bf16)lo, (__bf16)hi};
        return __builtin_bit_cast(uint32_t, v);
    } else {
        return DT::pack2(lo, hi);
    }
}

// A thread's units of a head.  Unit u is V elements of each half that turn against each
// other (half layout), V elements of V / 2 interleaved pairs (or one pair, two
// elements, when V is 1), or V elements that do not turn.  kVec: V elements are 16 bytes
// and every address is a multiple of that; V is 1 otherwise.  kLanes > 0 (with kVec and K = 1):
// every element turns, in half layout, and each of kLanes lanes has a unit, so nothing of a
// unit is a question at run time and sums need no branch (forward, 32 + 8 heads of 128: one row 3.0 against
// 3.4 us, 4096 rows 16.6 against 17.1; the gradients gain nothing, and have no such form).
template <typename DT, bool kVec, int K, int kLanes>
struct HeadUnits {
    using T = typename DT::storage;
    static constexpr int V = kVec ? 16 / DT::kBytes : 1;
    static constexpr bool kWhole = kLanes > 0;
    using Piece = std::conditional_t<kVec, uint4, T>;
    int at[K], next[K];     // first element, distance of the second piece (0: none)
    int unit[K];            // -1: none
    bool turns[K];

    __device__ __forceinline__ void init(const NormRopeArgs& a, int lane) {
        const int half = a.rot / 2;
        const int n_turned = a.interleaved ? (kVec ? a.rot / V : half) : half / V;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = lane + k * a.lanes;
            unit[k] = kWhole || i < a.units ? i : -1;
            turns[k] = kWhole || i < n_turned;
            if (kWhole) at[k] = i * V;
            else at[k] = !turns[k] ? a.rot + (i - n_turned) * V : a.interleaved ? (kVec ? i * V : 2 * i) : i * V;
            if (kWhole) next[k] = half;
            else next[k] = !turns[k] ? 0 : a.interleaved ? (kVec ? 0 : 1) : half;
        }
    }
    __device__ __forceinline__ bool here(int k) const { return kWhole || unit[k] >= 0; }
    __device__ __forceinline__ bool turned(int k) const { return kWhole || turns[k]; }
    __device__ __forceinline__ bool second(int k) const { return kWhole || next[k] != 0; }
    // Both pieces of every unit from a head's first element; absent ones are zeros.
    struct Raw {
        Piece x[K], y[K];
    };
    __device__ __forceinline__ void load(const T* p, Raw& r) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (kWhole) {
                r.x[k] = *reinterpret_cast<const Piece*>(p + at[k]);
                r.y[k] = *reinterpret_cast<const Piece*>(p + at[k] + next[k]);
            } else {
                r.x[k] = Piece{};
                r.y[k] = Piece{};
                if (!here(k)) continue;
                r.x[k] = *reinterpret_cast<const Piece*>(p + at[k]);
                if (second(k)) r.y[k] = *reinterpret_cast<const Piece*>(p + at[k] + next[k]);
            }
        }
    }
    // A weight's pieces that stay packed: unpacked again for each head, or they would be 16 registers
    // more.
    __device__ static __forceinline__ void stay_packed(Raw& r) {
        if constexpr (V == 8) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                asm volatile("" : "+v"(r.x[k].x), "+v"(r.x[k].y), "+v"(r.x[k].z), "+v"(r.x[k].w), "+v"(r.y[k].x),
                             "+v"(r.y[k].y), "+v"(r.y[k].z), "+v"(r.y[k].w));
        }
    }
    __device__ static __forceinline__ void unpack(const Piece& p, float* f) {
        if constexpr (kVec) DT::unpack(p, f);
        else f[0] = DT::load1(&p);
    }
    __device__ static __forceinline__ uint4 pack(const float* f) {
        if constexpr (V == 8)
            return make_uint4(norm_pack2<DT>(f[0], f[1]), norm_pack2<DT>(f[2], f[3]), norm_pack2<DT>(f[4], f[5]),
                              norm_pack2<DT>(f[6], f[7]));
        else return DT::pack(f);
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
            if (!here(k)) continue;
            if constexpr (kVec) {
                store16(p + at[k], pack(f[k]));
                if (second(k)) store16(p + at[k] + next[k], pack(f[k] + V));
            } else {
                p[at[k]] = DT::from_float(f[k][0]);
                if (second(k)) p[at[k] + next[k]] = DT::from_float(f[k][1]);
            }
        }
    }
    // Turns the units by the angles of their row (cosine and sine times the magnitude).
    __device__ __forceinline__ void turn(float (*f)[2 * V], const float* c, const float* s, bool pairs_inside,
                                         float sign) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!turned(k) || !here(k)) continue;
            if (kVec && !kWhole && pairs_inside) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float cc = c[unit[k] * (V / 2) + i], ss = s[unit[k] * (V / 2) + i] * sign;
                    const float x = f[k][2 * i], y = f[k][2 * i + 1];
                    f[k][2 * i] = x * cc - y * ss;
                    f[k][2 * i + 1] = y * cc + x * ss;
                }
            } else {
                float cc[V], ss[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if constexpr (kVec) {  // rot / 2 is a multiple of V here
                        if (i % 4 == 0) {
                            *reinterpret_cast<float4*>(cc + i) = *reinterpret_cast<const float4*>(c + unit[k] * V + i);
                            *reinterpret_cast<float4*>(ss + i) = *reinterpret_cast<const float4*>(s + unit[k] * V + i);
                        }
                    } else {
                        cc[i] = c[unit[k] * V + i];
                        ss[i] = s[unit[k] * V + i];
                    }
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = f[k][i], y = f[k][V + i], t = ss[i] * sign;
                    f[k][i] = x * cc[i] - y * t;
                    f[k][V + i] = y * cc[i] + x * t;
                }
            }
        }
    }
};

// The heads of a tensor's rows that a thread visits: item i is row i / heads, head i % heads,
// and a thread goes on by a workgroup's items at a time.
struct HeadWalk {
    int r, h, left, heads, rows_on, heads_on;
    __device__ __forceinline__ HeadWalk(int slot, int step, int n_rows, int n_heads) {
        heads = max(n_heads, 1);
        r = slot / heads;
        h = slot - r * heads;
        rows_on = step / heads;
        heads_on = step - rows_on * heads;
        left = n_heads > 0 ? n_rows : 0;
    }
    __device__ __forceinline__ bool here() const { return r < left; }
    __device__ __forceinline__ void go_on() {
        r += rows_on;
        h += heads_on;
        if (h >= heads) {
            h -= heads;
            ++r;
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
        // fraction of a turn in [-1/2, 1/2], times 2: sincospi's argument.  In float32 it is off by up to 2^-26, 1e-7
        // of the angle, which enters to first order: 2 pi cos of it into the sine and the reverse.
        const double t = pos * a.freq[j] * 0.15915494309189533577, turn = t - rint(t);
        const float near = (float)turn, off = 6.2831853f * (float)(turn - near);
        float sn, cs;
        sincospif(2.f * near, &sn, &cs);
        s_cos[i] = __builtin_fmaf(-sn, off, cs) * a.mag;
        s_sin[i] = __builtin_fmaf(cs, off, sn) * a.mag;
    }
}

template <typename DT, bool kVec, int K, int kLanes>
__global__ __launch_bounds__(kNormThreads, K == 1 ? 5 : 1) void norm_rope_kernel(NormRopeArgs a) {
    using Units = HeadUnits<DT, kVec, K, kLanes>;
    using T = typename DT::storage;
    constexpr int V = Units::V;
    __shared__ __align__(16) float s_cos[kNormAngles], s_sin[kNormAngles];
    const int blk = (int)(blockIdx.x / (unsigned)a.groups);
    const int grp = (int)(blockIdx.x - (unsigned)blk * a.groups);
    const int row0 = blk * a.rows_per_block;
    const int rows = min(a.rows_per_block, a.rows - row0);
    const int h_lo = grp * a.heads_per_group;
    const int h_hi = min(h_lo + a.heads_per_group, a.heads[0] + a.heads[1]);
    const int lanes = kLanes ? kLanes : a.lanes;
    const int lane = threadIdx.x & (lanes - 1), step = kNormThreads / lanes, half = a.rot / 2;
    const int slot = threadIdx.x / lanes;
    Units un;
    un.init(a, lane);

    // The group's heads of queries, then those of keys; the first loads of both go out ahead of the angles.
    const int lo[2] = {min(h_lo, a.heads[0]), max(h_lo - a.heads[0], 0)};
    const int hi[2] = {min(h_hi, a.heads[0]), max(h_hi - a.heads[0], 0)};
    HeadWalk walk[2] = {HeadWalk(slot, step, rows, hi[0] - lo[0]), HeadWalk(slot, step, rows, hi[1] - lo[1])};
    typename Units::Raw raw[2], wr[2];
    auto load = [&](int w, const HeadWalk& at) {
        un.load((const T*)a.in[w] + (long long)(row0 + at.r) * a.in_row[w] + (long long)(lo[w] + at.h) * a.in_head[w],
                raw[w]);
    };
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (!walk[w].here()) continue;
        load(w, walk[w]);
        if (a.weight[w]) un.load((const T*)a.weight[w], wr[w]);
    }
    norm_angles(a, row0, rows, s_cos, s_sin);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        while (walk[w].here()) {
            const HeadWalk at = walk[w];
            float f[K][2 * V];
            un.floats(raw[w], f);
            walk[w].go_on();
            if (walk[w].here()) load(w, walk[w]);  // the next head, behind this one's sums
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) ss += f[k][i] * f[k][i];
            const float rs = 1.f / sqrtf(head_sum(ss, lanes) * a.inv_D + a.eps);
            if (a.weight[w]) {
                float wf[K][2 * V];
                un.stay_packed(wr[w]);
                un.floats(wr[w], wf);
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
            un.turn(f, s_cos + at.r * half, s_sin + at.r * half, a.interleaved, 1.f);
            un.store((T*)a.out[w] + (long long)(row0 + at.r) * a.out_row[w] + (long long)(lo[w] + at.h) * a.out_head[w],
                     f);
        }
    }
}

// Gradients.  The first a.split workgroups are the queries' and the others the keys'; one takes blocks of rows,
// every so many, and its threads keep the sums of the weight's gradient over all of them.  x stays packed
// and is unpacked twice: with that 128 registers hold all, 4 waves a SIMD.
template <typename DT, bool kVec, int K>
__global__ __launch_bounds__(kNormThreads, K == 1 ? 4 : 1) void norm_rope_grad_kernel(NormRopeArgs a) {
    using Units = HeadUnits<DT, kVec, K, 0>;
    using T = typename DT::storage;
    constexpr int V = Units::V;
    __shared__ __align__(16) float s_cos[kNormAngles], s_sin[kNormAngles];
    __shared__ float s_sum[kNormThreads / kWave * kNormMaxDim];
    const int lanes = a.lanes, lane = threadIdx.x & (lanes - 1), step = kNormThreads / lanes, half = a.rot / 2;
    const int slot = threadIdx.x / lanes, wave = threadIdx.x / kWave;
    const int w = (int)blockIdx.x >= a.split;
    const int first = (int)blockIdx.x - (w ? a.split : 0), on = w ? (int)gridDim.x - a.split : a.split;
    const int block_rows = w ? a.grad_rows[1] : a.grad_rows[0], heads = w ? a.heads[1] : a.heads[0];
    const T* in = (const T*)(w ? a.in[1] : a.in[0]);
    const T* grad = (const T*)(w ? a.grad[1] : a.grad[0]);
    const T* weight = (const T*)(w ? a.weight[1] : a.weight[0]);
    T* out = (T*)(w ? a.out[1] : a.out[0]);
    const long long in_row = w ? a.in_row[1] : a.in_row[0], in_head = w ? a.in_head[1] : a.in_head[0];
    const long long grad_row = w ? a.grad_row[1] : a.grad_row[0], grad_head = w ? a.grad_head[1] : a.grad_head[0];
    const long long out_row = w ? a.out_row[1] : a.out_row[0], out_head = w ? a.out_head[1] : a.out_head[0];
    Units un;
    un.init(a, lane);
    float acc[K][2 * V] = {};
    typename Units::Raw wr;
    if (weight) un.load(weight, wr);
    for (long long row0 = (long long)first * block_rows; row0 < a.rows; row0 += (long long)on * block_rows) {
        const int rows = (int)min((long long)block_rows, a.rows - row0);
        HeadWalk walk(slot, step, rows, heads);
        typename Units::Raw rx, rg;
        auto load = [&]() {
            un.load(in + (row0 + walk.r) * in_row + walk.h * in_head, rx);
            un.load(grad + (row0 + walk.r) * grad_row + walk.h * grad_head, rg);
        };
        if (walk.here()) load();
        __syncthreads();
        norm_angles(a, (int)row0, rows, s_cos, s_sin);
        __syncthreads();
        while (walk.here()) {
            const int r = walk.r, h = walk.h;
            typename Units::Raw px = rx;
            float x[K][2 * V], g[K][2 * V], wf[K][2 * V];
            un.floats(rg, g);
            walk.go_on();
            if (walk.here()) load();
            auto weights = [&]() {
                if (weight) {
                    un.stay_packed(wr);
                    un.floats(wr, wf);
                } else {
#pragma unroll
                    for (int k = 0; k < K; ++k)
#pragma unroll
                        for (int i = 0; i < 2 * V; ++i) wf[k][i] = 1.f;
                }
            };
            un.turn(g, s_cos + r * half, s_sin + r * half, a.interleaved, -1.f);
            un.floats(px, x);
            weights();
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) {
                    ss += x[k][i] * x[k][i];
                    dot += g[k][i] * wf[k][i] * x[k][i];
                }
            ss = head_sum(ss, lanes);
            dot = head_sum(dot, lanes);
            const float rs = 1.f / sqrtf(ss * a.inv_D + a.eps);
            const float back = rs * rs * (dot * a.inv_D);
            un.stay_packed(px);
            un.floats(px, x);
            weights();
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) {
                    acc[k][i] += g[k][i] * (x[k][i] * rs);
                    g[k][i] = rs * (g[k][i] * wf[k][i] - x[k][i] * back);
                }
            if (out) un.store(out + (row0 + r) * out_row + h * out_head, g);
        }
    }
    if (!(w ? a.sums[1] : a.sums[0])) return;
    // Over the workgroup's heads: those of a wave by lane moves, those of its waves through LDS.
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) {
            float t = acc[k][i];
            for (int m = lanes; m < kWave; m *= 2) t += __shfl_xor(t, m);
            if ((int)(threadIdx.x & (kWave - 1)) < lanes && un.here(k) && (i < V || un.second(k)))
                s_sum[wave * a.D + un.at[k] + (i < V ? i : un.next[k] + i - V)] = t;
        }
    __syncthreads();
    float* sum = a.partial + (long long)blockIdx.x * a.D;
    for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
        float t = s_sum[d];
#pragma unroll
        for (int v = 1; v < kNormThreads / kWave; ++v) t += s_sum[v * a.D + d];
        sum[d] = t;
    }
}

// The weights' gradients: sums of n partials per element, rounded once.  Workgroup (x, w) has
// 16 elements; thread (e, g) sums every 64th partial from g, eight loads at a time, then these are added in a fixed
// order, four of a wave by lane moves and the waves' sums by the first wave.  In float64: up to 1024 float32 steps
// would lose more than all sums before (1003 rows of 5 + 5 heads of 80: 1.8e-7 off, with float64 0.8e-7).
template <typename DT>
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* partial, void* dwq, void* dwk, int nq, int nk,
                                                         int D) {
    using T = typename DT::storage;
    __shared__ double s[16][16];
    const int w = blockIdx.y, e = threadIdx.x & 15, g = threadIdx.x / 16;
    const int d = blockIdx.x * 16 + e;
    T* out = (T*)(w ? dwk : dwq);
    if (!out) return;
    const int n = w ? nk : nq;
    if (w) partial += (long long)nq * D;
    double t = 0.0;
    for (int i0 = g; i0 < n; i0 += 64 * 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)  // in no branch, or each would be waited for by itself
            v[k] = partial[(long long)min(i0 + 64 * k, n - 1) * D + min(d, D - 1)];
#pragma unroll
        for (int k = 0; k < 8; ++k) t += i0 + 64 * k < n ? (double)v[k] : 0.0;
    }
    auto four = [](double x) {
        x += __shfl_xor(x, 16);
        return x + __shfl_xor(x, 32);
    };
    t = four(t);
    if ((g & 3) == 0) s[g / 4][e] = t;
    __syncthreads();
    if (g >= 4) return;
    t = four((s[4 * g][e] + s[4 * g + 1][e]) + (s[4 * g + 2][e] + s[4 * g + 3][e]));
    if (g == 0 && d < D) out[d] = DT::from_float((float)t);
}

}  // namespace sgmv

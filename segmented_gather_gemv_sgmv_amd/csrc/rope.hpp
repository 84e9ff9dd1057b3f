// rope.hpp -- rotary positions on q and k.
//
// Pair j of a head's first `rot` elements, (a, b) = (x[j], x[j + rot / 2]) in
// the half layout or (x[2 j], x[2 j + 1]) interleaved, is turned by the angle
// t = position * f_j and scaled by m:
//     a' = m (a cos t - b sin t),   b' = m (b cos t + a sin t);
// elements from `rot` on are copied.  The gradients turn back, by -t.
//
// Bound: HBM (each element is read once and written once, a handful of
// flops); at decode sizes the launch.  The angle needs more than float32:
// at position 10^5 its float32 product is already off by 2^-8 radians.  So
// the product is taken in float64 and reduced to a fraction of a turn there
// (one multiply, one round, one subtract), and only that fraction's sine
// and cosine are float32.  All heads of a row share its angles: a workgroup
// computes them once into LDS and then streams heads.
#pragma once

#include <type_traits>

#include "proj_plan.hpp"
#include "sgmv_device.hpp"

namespace sgmv {

struct RopeArgs {
    void* out[2];
    const void* in[2];
    long long in_row[2], in_head[2];    // strides in elements; the last dim's is 1
    long long out_row[2], out_head[2];
    const void* positions;              // [rows], int32 or int64
    int wide_positions;                 // int64
    const double* freq;                 // [rot / 2], radians per position
    float mag, sign;
    int rows, heads[2], D, rot;
    int groups, heads_per_group;        // head groups of a row, one workgroup each
    int units;                          // work units per head
    uint32_t units_magic;               // ceil(2^32 / units)
    int interleaved;
};

// n / units for n < 2^16: exact with magic = ceil(2^32 / units) while
// n * (units * magic - 2^32) < 2^32, i.e. n * units < 2^32.
__device__ __forceinline__ int rope_div(int n, uint32_t magic, int units) {
    return units == 1 ? n : (int)__umulhi((uint32_t)n, magic);
}

// A unit is V elements copied, V elements of V / 2 interleaved pairs (or one
// pair), or V pairs of the half layout (a piece of the lower and its piece of
// the upper half).  kVec: V elements are 16 bytes; every stride, base address, D
// and (half layout) rot / 2, (interleaved) rot is a multiple of V.  Otherwise
// V is 1.
//
// Every thread asks for its (up to U) units before it computes an angle, so the
// angles' latency (position, frequency, float64 product, sine and cosine) hides
// behind the loads'.  8191 rows of 32 + 8 heads of 80, 32 turned, bf16, forward,
// 105 MB: 53 us cold with the loads after the angles, 28 us this way.
template <typename DT, bool kVec, int U>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    using T = typename DT::storage;
    constexpr int V = kVec ? 16 / DT::kBytes : 1;
    using Piece = std::conditional_t<kVec, uint4, T>;
    __shared__ float s_cos[kRopeMaxDim / 2], s_sin[kRopeMaxDim / 2];
    const int row = (int)(blockIdx.x / (unsigned)a.groups);
    const int grp = (int)(blockIdx.x - (unsigned)row * a.groups);
    const int tid = threadIdx.x;
    const int half = a.rot / 2;
    const int h_lo = grp * a.heads_per_group;
    const int h_hi = min(h_lo + a.heads_per_group, a.heads[0] + a.heads[1]);
    const int turned = a.interleaved ? (kVec ? a.rot / V : half) : half / V;
    const int total = (h_hi - h_lo) * a.units;

    // Unit e: its source and destination (elements from it on), its second
    // piece's distance (half layout and single interleaved pairs), its index.
    struct Unit {
        const T* src;
        T* dst;
        int second, u;  // second: 0 if there is none
    };
    auto locate = [&](int e) {
        const int hh = rope_div(e, a.units_magic, a.units);
        const int u = e - hh * a.units;
        int h = h_lo + hh;
        const int w = h >= a.heads[0];
        if (w) h -= a.heads[0];
        Unit t;
        t.u = u;
        int at;
        if (u >= turned) {
            at = a.rot + (u - turned) * V;
            t.second = 0;
        } else if (a.interleaved) {
            at = kVec ? u * V : 2 * u;
            t.second = kVec ? 0 : 1;
        } else {
            at = u * V;
            t.second = half;
        }
        t.src = (const T*)a.in[w] + (long long)row * a.in_row[w] + (long long)h * a.in_head[w] + at;
        t.dst = (T*)a.out[w] + (long long)row * a.out_row[w] + (long long)h * a.out_head[w] + at;
        return t;
    };
    auto load = [](const T* p) { return *reinterpret_cast<const Piece*>(p); };
    auto unpack = [](const Piece& p, float* f) {
        if constexpr (kVec) DT::unpack(p, f);
        else f[0] = DT::load1(&p);
    };
    auto store = [](T* p, const float* f) {
        if constexpr (kVec) store16(p, DT::pack(f));
        else *p = DT::from_float(f[0]);
    };

    Unit unit[U];
    Piece x[U], y[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int e = tid + k * kRopeThreads;
        if (e < total) {
            unit[k] = locate(e);
            x[k] = load(unit[k].src);
            if (unit[k].second) y[k] = load(unit[k].src + unit[k].second);
        }
    }
    const double pos = a.wide_positions ? (double)((const long long*)a.positions)[row]
                                        : (double)((const int*)a.positions)[row];
    for (int j = tid; j < half; j += kRopeThreads) {
        // fraction of a turn in [-1/2, 1/2], times 2: sincospi's argument
        const double t = pos * a.freq[j] * 0.15915494309189533577;
        const float r = 2.f * (float)(t - rint(t));
        float s, c;
        sincospif(r, &s, &c);
        s_cos[j] = c * a.mag;
        s_sin[j] = s * a.mag * a.sign;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (tid + k * kRopeThreads >= total) break;
        const Unit& t = unit[k];
        if (t.u >= turned) {
            *reinterpret_cast<Piece*>(t.dst) = x[k];
        } else if (kVec && a.interleaved) {
            float f[V], o[V];
            unpack(x[k], f);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float c = s_cos[t.u * (V / 2) + i], s = s_sin[t.u * (V / 2) + i];
                o[2 * i] = f[2 * i] * c - f[2 * i + 1] * s;
                o[2 * i + 1] = f[2 * i + 1] * c + f[2 * i] * s;
            }
            store(t.dst, o);
        } else {
            float f[V], g[V], o[V], p[V];
            unpack(x[k], f);
            unpack(y[k], g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float c = s_cos[t.u * V + i], s = s_sin[t.u * V + i];
                o[i] = f[i] * c - g[i] * s;
                p[i] = g[i] * c + f[i] * s;
            }
            store(t.dst, o);
            store(t.dst + t.second, p);
        }
    }
}

}  // namespace sgmv

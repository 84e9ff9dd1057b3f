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

#include "proj_device.hpp"

namespace sgmv {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxRot = 1024;

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

// kVec: V = 16 bytes of elements move at a time; every stride, base address,
// D and (half layout) rot / 2, (interleaved) rot is a multiple of V.
// Otherwise units are single pairs and single copied elements.
template <typename DT, bool kVec>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    using T = typename DT::storage;
    constexpr int V = kVec ? 16 / DT::kBytes : 1;
    __shared__ float s_cos[kRopeMaxRot / 2], s_sin[kRopeMaxRot / 2];
    const int row = (int)(blockIdx.x / (unsigned)a.groups);
    const int grp = (int)(blockIdx.x - (unsigned)row * a.groups);
    const int tid = threadIdx.x;
    const int half = a.rot / 2;
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

    // Units of a head: rotated ones first (half: V pairs, a piece of the lower
    // and its piece of the upper half; interleaved: V / 2 pairs, or one), then
    // copied pieces of V elements.
    const int h_lo = grp * a.heads_per_group;
    const int h_hi = min(h_lo + a.heads_per_group, a.heads[0] + a.heads[1]);
    const int turned = a.interleaved ? (kVec ? a.rot / V : half) : half / V;
    const int total = (h_hi - h_lo) * a.units;
    for (int e = tid; e < total; e += kRopeThreads) {
        const int hh = rope_div(e, a.units_magic, a.units);
        const int u = e - hh * a.units;
        int h = h_lo + hh;
        const int w = h >= a.heads[0];
        if (w) h -= a.heads[0];
        const T* src = (const T*)a.in[w] + (long long)row * a.in_row[w] + (long long)h * a.in_head[w];
        T* dst = (T*)a.out[w] + (long long)row * a.out_row[w] + (long long)h * a.out_head[w];
        if (u >= turned) {
            const int c = a.rot + (u - turned) * V;
            if constexpr (kVec) store16(dst + c, load16(src + c));
            else dst[c] = src[c];
        } else if (a.interleaved) {
            if constexpr (kVec) {
                float f[V], o[V];
                DT::unpack(load16(src + u * V), f);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float c = s_cos[u * (V / 2) + i], s = s_sin[u * (V / 2) + i];
                    o[2 * i] = f[2 * i] * c - f[2 * i + 1] * s;
                    o[2 * i + 1] = f[2 * i + 1] * c + f[2 * i] * s;
                }
                store16(dst + u * V, DT::pack(o));
            } else {
                const float x = DT::load1(src + 2 * u), y = DT::load1(src + 2 * u + 1);
                dst[2 * u] = DT::from_float(x * s_cos[u] - y * s_sin[u]);
                dst[2 * u + 1] = DT::from_float(y * s_cos[u] + x * s_sin[u]);
            }
        } else {
            if constexpr (kVec) {
                float x[V], y[V], o[V], p[V];
                DT::unpack(load16(src + u * V), x);
                DT::unpack(load16(src + half + u * V), y);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float c = s_cos[u * V + i], s = s_sin[u * V + i];
                    o[i] = x[i] * c - y[i] * s;
                    p[i] = y[i] * c + x[i] * s;
                }
                store16(dst + u * V, DT::pack(o));
                store16(dst + half + u * V, DT::pack(p));
            } else {
                const float x = DT::load1(src + u), y = DT::load1(src + half + u);
                dst[u] = DT::from_float(x * s_cos[u] - y * s_sin[u]);
                dst[half + u] = DT::from_float(y * s_cos[u] + x * s_sin[u]);
            }
        }
    }
}

}  // namespace sgmv

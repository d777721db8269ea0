// Group norm with an activation, channels last: x [N, L, C], G groups of D = C / G
// channels; statistics of each (sample, group) over its L positions and D channels.
//   xhat = (x - mean) rstd,  z = xhat w + b,  y = act(z), or z act(gate) with a gate
// Backward, for dy:
//   dz = dy act'(z)  (with a gate: dy act(gate), and dgate = dy z act'(gate))
//   dw = sum dz xhat,  db = sum dz  over samples and positions
//   t = dz w,  dx = rstd (t - m1 - xhat m2),  m1, m2 = means of t and t xhat over the group
// All arithmetic is in fp32; y, dx and dgate are rounded once, at the store.
//
// Three forms.  Rows (L = 1, D in whole 16-byte vectors): a group is D contiguous elements
// held in the registers of part of a warp, one read and one write of every element.
// Cluster (several positions of whole groups that fit the shared memory of up to eight CTAs):
// a thread-block cluster holds one sample's block of groups, and its CTAs exchange their sums
// through distributed shared memory; one kernel, one read of every element.
// Positions (any L, C, D): sums of row tiles, then a second kernel that joins them per group
// and reads x again (from L2 where it fits).
#pragma once

#include <algorithm>

#include <cooperative_groups.h>

#include "kda_common.cuh"
#include "kda_launch.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace norm {

// ------------------------------------------------------------------ element access

template <typename T, int VEC>
struct Vec;   // VEC consecutive elements, loaded and stored as one access
template <>
struct Vec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void open(const uint4 &r, float (&f)[8]) {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 close(const float (&f)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Vec<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ void open(const float4 &r, float (&f)[4]) {
        f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
    }
    static __device__ __forceinline__ float4 close(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Vec<__nv_bfloat16, 1> {
    using Raw = __nv_bfloat16;
    static __device__ __forceinline__ void open(const Raw &r, float (&f)[1]) { f[0] = __bfloat162float(r); }
    static __device__ __forceinline__ Raw close(const float (&f)[1]) { return __float2bfloat16_rn(f[0]); }
};
template <>
struct Vec<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ void open(const Raw &r, float (&f)[1]) { f[0] = r; }
    static __device__ __forceinline__ Raw close(const float (&f)[1]) { return f[0]; }
};
template <typename T>
constexpr int vec_of() { return 16 / (int)sizeof(T); }
// A 16-byte vector as pairs, for two operations an instruction
template <typename T>
__device__ __forceinline__ void open_pairs(const typename Vec<T, vec_of<T>()>::Raw &r, float2 (&f)[vec_of<T>() / 2]) {
    float e[vec_of<T>()];
    Vec<T, vec_of<T>()>::open(r, e);
#pragma unroll
    for (int i = 0; i < vec_of<T>() / 2; ++i) f[i] = make_float2(e[2 * i], e[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ typename Vec<T, vec_of<T>()>::Raw close_pairs(const float2 (&f)[vec_of<T>() / 2]) {
    float e[vec_of<T>()];
#pragma unroll
    for (int i = 0; i < vec_of<T>() / 2; ++i) {
        e[2 * i] = f[i].x;
        e[2 * i + 1] = f[i].y;
    }
    return Vec<T, vec_of<T>()>::close(e);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[VEC]) {
    Vec<T, VEC>::open(*reinterpret_cast<const typename Vec<T, VEC>::Raw *>(p), f);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[VEC]) {
    *reinterpret_cast<typename Vec<T, VEC>::Raw *>(p) = Vec<T, VEC>::close(f);
}

// 16-byte access to data that is touched once.
template <typename Raw, typename T>
__device__ __forceinline__ Raw ld_raw(const T *p) {
    return __ldcs(reinterpret_cast<const Raw *>(p));
}
template <typename Raw, typename T>
__device__ __forceinline__ void st_raw(T *p, const Raw &v) {
    __stcs(reinterpret_cast<Raw *>(p), v);
}

// ------------------------------------------------------------------ activations

// 1 / (1 + e^-x).  The hardware exponential's error (about |x| 2^-23 relative) and reciprocal's
// are far inside a bf16 step; fp32 tensors take the full-precision exponential.
template <typename T>
__device__ __forceinline__ float logistic(float x) {
    if (sizeof(T) == 4) return __fdividef(1.f, 1.f + expf(-x));   // e = inf gives 0
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <typename T, int ACT>
__device__ __forceinline__ float act(float x) {
    return ACT == KDA_ACT_NONE ? x : ACT == KDA_ACT_SILU ? x * logistic<T>(x) : logistic<T>(x);
}
// value and slope
template <typename T, int ACT>
__device__ __forceinline__ float2 act2(float x) {
    if (ACT == KDA_ACT_NONE) return make_float2(x, 1.f);
    const float p = logistic<T>(x);
    return ACT == KDA_ACT_SILU ? make_float2(x * p, p * fmaf(x, 1.f - p, 1.f)) : make_float2(p, p * (1.f - p));
}

// one element: z and dy (and the gate's value) -> dz (and dgate)
template <typename T, int ACT, bool GATE>
__device__ __forceinline__ float back_act(float z, float dy, float gate, float &dgate) {
    if (GATE) {
        const float2 a = act2<T, ACT>(gate);
        dgate = dy * z * a.y;
        return dy * a.x;
    }
    return dy * act2<T, ACT>(z).y;
}

// sum over the `lanes` (a power of two) neighbouring lanes of a warp
__device__ __forceinline__ float lane_sum(float x, int lanes) {
    for (int o = lanes >> 1; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// the same over LANES lanes, unrolled; LANES = 0: `lanes`
template <int LANES>
__device__ __forceinline__ float group_sum(float x, int lanes) {
    if constexpr (LANES == 0) {
        return lane_sum(x, lanes);
    } else {
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    }
}

// ------------------------------------------------------------------ rows form

constexpr int kThreads = 256;

struct RowsGeo {
    long long rows;   // N G
    int G, D;
    int lanes;        // lanes of a row: a power of two, D <= lanes NV VEC
    int step;         // rows between two rows of one lane group: a multiple of G
};

// Resident CTAs per SM that the rows kernels are launched and bounded for: as many as leave
// the registers for NV vectors of every tensor.
constexpr int rows_ctas(int nv, bool backward) {
    return backward ? (nv == 1 ? 2 : 1) : nv == 1 ? 3 : nv == 2 ? 2 : 1;
}

// What a lane keeps of its group: weights, and which of its vectors exist.
template <typename T, int NV, int LANES>
struct Lane {
    static constexpr int VEC = vec_of<T>(), P = VEC / 2;
    int sl, g, lanes, D;
    long long sub;
    float2 wt[NV][P], bs[NV][P];
    __device__ __forceinline__ Lane(const RowsGeo &r, const float *weight, const float *bias)
        : lanes(LANES ? LANES : r.lanes), D(LANES ? LANES * NV * VEC : r.D) {
        const int per = kThreads / lanes;
        sl = threadIdx.x & (lanes - 1);
        sub = (long long)blockIdx.x * per + threadIdx.x / lanes;
        g = (int)(sub % r.G);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const long long c = (long long)g * D + at(j) + 2 * e;
                wt[j][e] = on(j) && weight ? make_float2(weight[c], weight[c + 1]) : both(1.f);
                bs[j][e] = on(j) && bias ? make_float2(bias[c], bias[c + 1]) : both(0.f);
            }
    }
    __device__ __forceinline__ int at(int j) const { return (sl + j * lanes) * VEC; }
    __device__ __forceinline__ bool on(int j) const { return LANES || at(j) < D; }
    // the first row of the warp: whole lane groups leave a loop together with their warp's others
    __device__ __forceinline__ long long warp_first() const {
        return (long long)blockIdx.x * (kThreads / lanes) + (threadIdx.x & ~31) / lanes;
    }
};

// Rows of NV vectors a lane, U at a time.  A lane group keeps one group index g, so its weights
// stay in registers.  LANES > 0: that many lanes hold a row exactly.  Arithmetic runs in pairs:
// at 8 bytes an element and less the instructions, not the bytes, are what takes the time
// (36 instructions an element took 48 us where the bytes take 31).
template <typename T, int NV, int LANES, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads, rows_ctas(NV, false))
rows_forward_kernel(RowsGeo r, const T *__restrict__ x, const float *__restrict__ weight,
                    const float *__restrict__ bias, const T *__restrict__ gate, T *__restrict__ y,
                    float *__restrict__ mean, float *__restrict__ rstd, float eps) {
    constexpr int U = NV == 1 ? 2 : 1, P = vec_of<T>() / 2;
    using Raw = typename Vec<T, vec_of<T>()>::Raw;
    const Lane<T, NV, LANES> l(r, weight, bias);
    const float inv = 1.f / l.D;
    struct Rows {
        Raw x[U][NV], g[U][NV];
    };
    auto fetch = [&](Rows &n, long long base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // behind the last row it is read again
            const long long row = min(l.sub + base + (long long)u * r.step, r.rows - 1);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!LANES) n.x[u][j] = n.g[u][j] = Raw();
                if (l.on(j)) {
                    n.x[u][j] = ld_raw<Raw>(x + row * l.D + l.at(j));
                    if (GATE) n.g[u][j] = ld_raw<Raw>(gate + row * l.D + l.at(j));
                }
            }
        }
    };
    auto work = [&](const Rows &c, long long base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = l.sub + base + (long long)u * r.step;
            float2 f[NV][P], a = both(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                open_pairs<T>(c.x[u][j], f[j]);
#pragma unroll
                for (int e = 0; e < P; ++e) a = ptx::add2(a, f[j][e]);   // lanes that hold nothing add zeros
            }
            const float m = group_sum<LANES>(a.x + a.y, l.lanes) * inv;
            a = both(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    f[j][e] = ptx::add2(f[j][e], both(-m));
                    if (l.on(j)) a = ptx::fma2(f[j][e], f[j][e], a);
                }
            const float rs = rsqrtf(group_sum<LANES>(a.x + a.y, l.lanes) * inv + eps);
            if (row >= r.rows) continue;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!l.on(j)) continue;
                float2 gv[P], out[P];
                if (GATE) open_pairs<T>(c.g[u][j], gv);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const float2 z = ptx::fma2(ptx::mul2(f[j][e], both(rs)), l.wt[j][e], l.bs[j][e]);
                    const float2 on = GATE ? gv[e] : z, v = make_float2(act<T, ACT>(on.x), act<T, ACT>(on.y));
                    out[e] = GATE ? ptx::mul2(z, v) : v;
                }
                st_raw(y + row * l.D + l.at(j), close_pairs<T>(out));
            }
            if (l.sl == 0) {
                mean[row] = m;
                rstd[row] = rs;
            }
        }
    };
    // two sets of rows in turn: one is in flight while the other is worked on
    Rows a, b;
    const long long stride = (long long)r.step * U;
    fetch(a, 0);
    for (long long base = 0; l.warp_first() + base < r.rows; base += 2 * stride) {
        fetch(b, base + stride);
        work(a, base);
        fetch(a, base + 2 * stride);
        work(b, base + stride);
    }
}

// part: [step / G][2][C] sums of dz xhat and dz over each lane group's rows.  The next rows'
// loads are in flight behind the ones it works on.
template <typename T, int NV, int LANES, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads, rows_ctas(NV, true))
rows_backward_kernel(RowsGeo r, const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
                     const float *__restrict__ rstd, const float *__restrict__ weight,
                     const float *__restrict__ bias, const T *__restrict__ gate, T *__restrict__ dx,
                     T *__restrict__ dgate, float *__restrict__ part) {
    let_next_start();
    constexpr int U = NV == 1 ? 2 : 1, P = vec_of<T>() / 2;
    using Raw = typename Vec<T, vec_of<T>()>::Raw;
    const Lane<T, NV, LANES> l(r, weight, bias);
    const float inv = 1.f / l.D;
    float2 dw[NV][P], db[NV][P];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < P; ++e) dw[j][e] = db[j][e] = both(0.f);
    struct Rows {
        Raw x[U][NV], y[U][NV], g[U][NV];
        float m[U], rs[U];
    };
    auto fetch = [&](Rows &n, long long base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = min(l.sub + base + (long long)u * r.step, r.rows - 1);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!LANES) n.x[u][j] = n.y[u][j] = n.g[u][j] = Raw();
                if (l.on(j)) {
                    n.x[u][j] = ld_raw<Raw>(x + row * l.D + l.at(j));
                    n.y[u][j] = ld_raw<Raw>(dy + row * l.D + l.at(j));
                    if (GATE) n.g[u][j] = ld_raw<Raw>(gate + row * l.D + l.at(j));
                }
            }
            n.m[u] = mean[row];
            n.rs[u] = rstd[row];
        }
    };
    auto work = [&](const Rows &c, long long base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = l.sub + base + (long long)u * r.step;
            const bool in = row < r.rows;
            const float m = c.m[u], rs = c.rs[u];
            float2 xh[NV][P], t[NV][P], s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float2 dv[P], gv[P], dg[P];
                open_pairs<T>(c.x[u][j], xh[j]);
                open_pairs<T>(c.y[u][j], dv);
                if (GATE) open_pairs<T>(c.g[u][j], gv);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    float2 h = ptx::mul2(ptx::add2(xh[j][e], both(-m)), both(rs));
                    const float2 z = ptx::fma2(h, l.wt[j][e], l.bs[j][e]);
                    float2 dz;
                    if (GATE) {
                        const float2 p = act2<T, ACT>(gv[e].x), q = act2<T, ACT>(gv[e].y);
                        dg[e] = ptx::mul2(ptx::mul2(dv[e], z), make_float2(p.y, q.y));
                        dz = ptx::mul2(dv[e], make_float2(p.x, q.x));
                    } else {
                        dz = ptx::mul2(dv[e], make_float2(act2<T, ACT>(z.x).y, act2<T, ACT>(z.y).y));
                    }
                    if (!in) dz = h = both(0.f);   // no row: what was read is another group's
                    xh[j][e] = h;
                    t[j][e] = ptx::mul2(dz, l.wt[j][e]);
                    dw[j][e] = ptx::fma2(dz, h, dw[j][e]);
                    db[j][e] = ptx::add2(db[j][e], dz);
                    s1 = ptx::add2(s1, t[j][e]);
                    s2 = ptx::fma2(t[j][e], h, s2);
                }
                if (GATE && in && l.on(j)) st_raw(dgate + row * l.D + l.at(j), close_pairs<T>(dg));
            }
            const float m1 = group_sum<LANES>(s1.x + s1.y, l.lanes) * inv;
            const float m2 = group_sum<LANES>(s2.x + s2.y, l.lanes) * inv;
            if (!in) continue;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!l.on(j)) continue;
                float2 out[P];
#pragma unroll
                for (int e = 0; e < P; ++e)
                    out[e] = ptx::mul2(both(rs), ptx::fma2(xh[j][e], both(-m2), ptx::add2(t[j][e], both(-m1))));
                st_raw(dx + row * l.D + l.at(j), close_pairs<T>(out));
            }
        }
    };
    // two sets of rows in turn, so that none is copied
    Rows a, b;
    const long long stride = (long long)r.step * U;
    fetch(a, 0);
    for (long long base = 0; l.warp_first() + base < r.rows; base += 2 * stride) {
        fetch(b, base + stride);
        work(a, base);
        fetch(a, base + 2 * stride);
        work(b, base + stride);
    }
    const long long C = (long long)r.G * l.D;
    float *p = part + (l.sub / r.G) * 2 * C + (long long)l.g * l.D;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (l.on(j))
#pragma unroll
            for (int e = 0; e < P; e += 2) {
                const int d = l.at(j) + 2 * e;
                store4(p + d, make_float4(dw[j][e].x, dw[j][e].y, dw[j][e + 1].x, dw[j][e + 1].y));
                store4(p + C + d, make_float4(db[j][e].x, db[j][e].y, db[j][e + 1].x, db[j][e + 1].y));
            }
}

// ------------------------------------------------------------------ positions form

// A CTA takes one row tile of one sample and one block of at most 256 vectors of channels:
// blockIdx.x = n tiles + tile, blockIdx.y = channel block.
struct PosGeo {
    int N, L, C, G, D;
    int tiles, tile_rows;   // row tiles of a sample
    int cvecs;              // C / VEC
    int tpr;                // threads of one row: min(cvecs, 256); a CTA holds 256 / tpr rows at a time
    int Z;                  // channel blocks: ceil(cvecs / tpr)
    int span;               // channels of a block: tpr VEC
    int ZG;                 // channel blocks that a group can touch
    __device__ __forceinline__ int rows_of(int tile) const { return min(tile_rows, L - tile * tile_rows); }
};

// The channels of block z, and of them those of group g.
template <int VEC>
struct Block {
    int c0, c1, g0, g1;
    __device__ __forceinline__ Block(const PosGeo &p, int z) {
        c0 = z * p.tpr * VEC;
        c1 = min(p.C, c0 + p.tpr * VEC);
        g0 = c0 / p.D;
        g1 = (c1 - 1) / p.D;
    }
};
template <int VEC>
__device__ __forceinline__ int channels_in(const PosGeo &p, int z, int g) {
    const Block<VEC> b(p, z);
    return min(b.c1, (g + 1) * p.D) - max(b.c0, g * p.D);
}
__device__ __forceinline__ int first_block(const PosGeo &p, int g) { return g * p.D / p.span; }
// Partial of (n, g, tile) and the group's own block k, counted from its first: a group has places for
// the blocks that it touches only (for all blocks the workspace would grow with C^2 where groups are narrow)
__device__ __forceinline__ long long part_at(const PosGeo &p, int n, int g, int tile, int k) {
    return (((long long)n * p.G + g) * p.tiles + tile) * p.ZG + k;
}
// Which of group g's blocks block z, from channel c0 on, is: the first, unless g starts before it
__device__ __forceinline__ int own_block(const PosGeo &p, int z, int c0, int g) {
    return g * p.D >= c0 ? 0 : z - first_block(p, g);
}

// Lanes that work on one of `groups` groups: all 256 threads are busy with as many at once as fit a warp's shuffles.
__device__ __forceinline__ int lanes_for(int groups) {
    int lanes = 32;
    while (lanes > 1 && lanes * groups > kThreads) lanes >>= 1;
    return lanes;
}

// Moments pooled over `lanes` lanes: `each(f)` calls f(count, mean, m2) for the lane's parts, every
// time the same ones.  The mean of all first, then each part's squares around it: no division
// but one, and nothing that a large mean cancels.
template <typename Each>
__device__ __forceinline__ float2 pooled_moments(int lanes, float inv_count, Each &&each) {
    float s = 0.f, q = 0.f;
    each([&](float n, float m, float) { s = fmaf(n, m, s); });
    const float mean = lane_sum(s, lanes) * inv_count;
    each([&](float n, float m, float m2) {
        const float d = m - mean;
        q += fmaf(n * d, d, m2);
    });
    return make_float2(mean, lane_sum(q, lanes));
}

// Moments of a row tile and channel block for each group it touches: part[n][g][tile][z] =
// (mean, m2).  A thread takes eight rows of its channels at a time: their mean, then their
// centred squares, joined to what it has, so that no large mean cancels in a difference of sums.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) pos_moments_kernel(PosGeo p, const T *__restrict__ x,
                                                               float2 *__restrict__ part) {
    let_next_start();
    __shared__ float sm_m[VEC * kThreads], sm_q[VEC * kThreads];
    const int tile = blockIdx.x % p.tiles, n = blockIdx.x / p.tiles, z = blockIdx.y;
    const int rl = threadIdx.x / p.tpr, cl = threadIdx.x % p.tpr, rows = kThreads / p.tpr;
    const int r0 = tile * p.tile_rows, r1 = r0 + p.rows_of(tile);
    const int cv = z * p.tpr + cl;
    float mean[VEC] = {}, m2[VEC] = {}, cnt = 0.f;
    if (rl < rows && cv < p.cvecs)
        for (int r = r0 + rl; r < r1; r += 8 * rows) {
            float f[8][VEC];
            int k = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r + i * rows < r1) {
                    load_vec<T, VEC>(x + ((long long)n * p.L + r + i * rows) * p.C + (long long)cv * VEC, f[i]);
                    k = i + 1;
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) f[i][e] = 0.f;
                }
            const float nb = (float)k, ik = 1.f / nb, t = cnt + nb, fr = nb / t;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float s = 0.f, q = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s += f[i][e];
                const float mb = s * ik;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < k) q = fmaf(f[i][e] - mb, f[i][e] - mb, q);
                const float d = mb - mean[e];
                mean[e] = fmaf(d, fr, mean[e]);
                m2[e] += fmaf(d * d, cnt * fr, q);
            }
            cnt = t;
        }
    // entry (row lane, channel of the block): [row lane][tpr VEC]
    if (rl < rows)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sm_m[(rl * p.tpr + cl) * VEC + e] = mean[e];
            sm_q[(rl * p.tpr + cl) * VEC + e] = m2[e];
        }
    __syncthreads();
    const Block<VEC> b(p, z);
    const int lanes = lanes_for(b.g1 - b.g0 + 1), sl = threadIdx.x & (lanes - 1);
    // (a warp's lane groups stay together; those behind the last group work on it once more)
    for (int g0 = b.g0 + (int)(threadIdx.x & ~31) / lanes; g0 <= b.g1; g0 += kThreads / lanes) {
        const int g = min(g0 + (int)(threadIdx.x & 31) / lanes, b.g1);
        const int first = max(b.c0, g * p.D) - b.c0, w = channels_in<VEC>(p, z, g);
        const float2 v = pooled_moments(lanes, 1.f / ((float)(r1 - r0) * w), [&](auto &&f) {
            for (int ri = 0; ri < rows; ++ri) {
                // rows of row lane ri: r0 + ri, then every `rows`
                const float have = (float)max(0, (r1 - r0 - ri + rows - 1) / rows);
                for (int c = sl; c < w; c += lanes) {
                    const int at = ri * p.tpr * VEC + first + c;
                    f(have, sm_m[at], sm_q[at]);
                }
            }
        });
        if (sl == 0) part[part_at(p, n, g, tile, own_block(p, z, b.c0, g))] = v;
    }
}

// y from x and the partial moments.  Each CTA joins the moments of its groups (the CTAs of
// tile 0 store them), then runs down its rows.
template <typename T, int VEC, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads) pos_apply_kernel(PosGeo p, const T *__restrict__ x,
                                                             const float *__restrict__ weight,
                                                             const float *__restrict__ bias,
                                                             const T *__restrict__ gate, T *__restrict__ y,
                                                             const float2 *__restrict__ part,
                                                             float *__restrict__ mean, float *__restrict__ rstd,
                                                             float eps) {
    wait_for_previous();
    __shared__ float2 stat[VEC * kThreads];   // (mean, rstd) of the block's groups
    const int tile = blockIdx.x % p.tiles, n = blockIdx.x / p.tiles, z = blockIdx.y;
    const Block<VEC> b(p, z);
    const int lanes = lanes_for(b.g1 - b.g0 + 1), sl = threadIdx.x & (lanes - 1);
    for (int g0 = b.g0 + (int)(threadIdx.x & ~31) / lanes; g0 <= b.g1; g0 += kThreads / lanes) {
        const int g = min(g0 + (int)(threadIdx.x & 31) / lanes, b.g1);
        const int z0 = first_block(p, g), zn = ((g + 1) * p.D - 1) / p.span - z0 + 1;
        const float inv = 1.f / ((float)p.L * p.D);
        const float2 v = pooled_moments(lanes, inv, [&](auto &&f) {
            for (int k = 0; k < zn; ++k) {
                const float w = (float)channels_in<VEC>(p, z0 + k, g);
                const float2 *at = part + part_at(p, n, g, 0, k);
#pragma unroll 4
                for (int t = sl; t < p.tiles; t += lanes) {
                    const float2 u = at[(long long)t * p.ZG];
                    f(w * p.rows_of(t), u.x, u.y);
                }
            }
        });
        if (sl == 0) {
            const float rs = rsqrtf(v.y * inv + eps);
            stat[g - b.g0] = make_float2(v.x, rs);
            if (tile == 0 && z == z0) {
                mean[(long long)n * p.G + g] = v.x;
                rstd[(long long)n * p.G + g] = rs;
            }
        }
    }
    __syncthreads();
    const int rl = threadIdx.x / p.tpr, cl = threadIdx.x % p.tpr, rows = kThreads / p.tpr;
    const int r0 = tile * p.tile_rows, r1 = r0 + p.rows_of(tile);
    const int cv = z * p.tpr + cl;
    if (rl >= rows || cv >= p.cvecs) return;
    float m[VEC], s[VEC], o[VEC];   // z = (x - m) s + o
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int c = cv * VEC + e;
        const float2 v = stat[c / p.D - b.g0];
        m[e] = v.x;
        s[e] = v.y * (weight ? weight[c] : 1.f);
        o[e] = bias ? bias[c] : 0.f;
    }
    for (int r = r0 + rl; r < r1; r += 4 * rows) {
        float f[4][VEC], gv[4][VEC];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r + i * rows < r1) {
                const long long at = ((long long)n * p.L + r + i * rows) * p.C + (long long)cv * VEC;
                load_vec<T, VEC>(x + at, f[i]);
                if (GATE) load_vec<T, VEC>(gate + at, gv[i]);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r + i * rows < r1) {
                float out[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float zz = fmaf(f[i][e] - m[e], s[e], o[e]);
                    out[e] = GATE ? zz * act<T, ACT>(gv[i][e]) : act<T, ACT>(zz);
                }
                store_vec<T, VEC>(y + ((long long)n * p.L + r + i * rows) * p.C + (long long)cv * VEC, out);
            }
    }
}

// Per-channel values of one thread of the backward kernels
template <int VEC>
struct Affine {
    float m[VEC], rs[VEC], wt[VEC], bs[VEC];
    __device__ __forceinline__ Affine(const PosGeo &p, int n, int cv, const float *mean, const float *rstd,
                                      const float *weight, const float *bias) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = cv * VEC + e;
            const long long i = (long long)n * p.G + c / p.D;
            m[e] = mean[i];
            rs[e] = rstd[i];
            wt[e] = weight ? weight[c] : 1.f;
            bs[e] = bias ? bias[c] : 0.f;
        }
    }
};

// (Launch bounds of both backward kernels: where channels are taken one by one the registers are kept to what
// leaves as many CTAs an SM as loads need in flight; 8192 x 41 heads of 100 channels, bf16: 1.20 ms, without 1.31.)
// Backward: sums of a row tile.  Per channel chan[n][tile][c] = (sum dz xhat, sum dz); per
// group part[n][g][tile][z] = (sum w dz, sum w dz xhat).  dgate is written here.
template <typename T, int VEC, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads, VEC == 1 && !GATE ? (sizeof(T) == 2 ? 8 : 5) : 0) pos_back_sums_kernel(
    PosGeo p, const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
    const float *__restrict__ rstd, const float *__restrict__ weight, const float *__restrict__ bias,
    const T *__restrict__ gate, T *__restrict__ dgate, float2 *__restrict__ chan, float2 *__restrict__ part) {
    let_next_start();
    __shared__ float sm_w[VEC * kThreads], sm_b[VEC * kThreads];
    const int tile = blockIdx.x % p.tiles, n = blockIdx.x / p.tiles, z = blockIdx.y;
    const int rl = threadIdx.x / p.tpr, cl = threadIdx.x % p.tpr, rows = kThreads / p.tpr;
    const int r0 = tile * p.tile_rows, r1 = r0 + p.rows_of(tile);
    const int cv = z * p.tpr + cl;
    const bool on = rl < rows && cv < p.cvecs;
    float dw[VEC] = {}, db[VEC] = {};
    if (on) {
        const Affine<VEC> a(p, n, cv, mean, rstd, weight, bias);
        for (int r = r0 + rl; r < r1; r += 2 * rows) {
            float f[2][VEC], dv[2][VEC], gv[2][VEC];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (r + i * rows < r1) {
                    const long long at = ((long long)n * p.L + r + i * rows) * p.C + (long long)cv * VEC;
                    load_vec<T, VEC>(x + at, f[i]);
                    load_vec<T, VEC>(dy + at, dv[i]);
                    if (GATE) load_vec<T, VEC>(gate + at, gv[i]);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (r + i * rows < r1) {
                    float dg[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float h = (f[i][e] - a.m[e]) * a.rs[e];
                        const float zz = fmaf(h, a.wt[e], a.bs[e]);
                        const float dz = back_act<T, ACT, GATE>(zz, dv[i][e], GATE ? gv[i][e] : 0.f, dg[e]);
                        dw[e] = fmaf(dz, h, dw[e]);
                        db[e] += dz;
                    }
                    if (GATE)
                        store_vec<T, VEC>(dgate + ((long long)n * p.L + r + i * rows) * p.C + (long long)cv * VEC, dg);
                }
        }
    }
    if (rl < rows)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sm_w[(rl * p.tpr + cl) * VEC + e] = dw[e];
            sm_b[(rl * p.tpr + cl) * VEC + e] = db[e];
        }
    __syncthreads();
    // the row lanes of each channel, in order; the sums stay in row lane 0's entries
    const Block<VEC> b(p, z);
    const int span = p.tpr * VEC;
    for (int i = threadIdx.x; i < b.c1 - b.c0; i += kThreads) {
        float2 v = make_float2(sm_w[i], sm_b[i]);
        for (int k = 1; k < rows; ++k) {
            v.x += sm_w[k * span + i];
            v.y += sm_b[k * span + i];
        }
        chan[((long long)n * p.tiles + tile) * p.C + b.c0 + i] = v;
        sm_w[i] = v.x;
        sm_b[i] = v.y;
    }
    __syncthreads();
    const int lanes = lanes_for(b.g1 - b.g0 + 1), sl = threadIdx.x & (lanes - 1);
    for (int g0 = b.g0 + (int)(threadIdx.x & ~31) / lanes; g0 <= b.g1; g0 += kThreads / lanes) {
        const int g = min(g0 + (int)(threadIdx.x & 31) / lanes, b.g1);
        const int first = max(b.c0, g * p.D), w = channels_in<VEC>(p, z, g);
        float s1 = 0.f, s2 = 0.f;
        for (int i = sl; i < w; i += lanes) {
            const float wt = weight ? weight[first + i] : 1.f;
            s1 = fmaf(wt, sm_b[first - b.c0 + i], s1);
            s2 = fmaf(wt, sm_w[first - b.c0 + i], s2);
        }
        s1 = lane_sum(s1, lanes);
        s2 = lane_sum(s2, lanes);
        if (sl == 0) part[part_at(p, n, g, tile, own_block(p, z, b.c0, g))] = make_float2(s1, s2);
    }
}

// dx; the CTAs behind the N tiles row tiles (blockIdx.y 0) sum dweight and dbias, 32 channels each.
template <typename T, int VEC, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads, VEC == 1 ? 5 : 0) pos_back_apply_kernel(
    PosGeo p, const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
    const float *__restrict__ rstd, const float *__restrict__ weight, const float *__restrict__ bias,
    const T *__restrict__ gate, T *__restrict__ dx, const float2 *__restrict__ chan, const float2 *__restrict__ part,
    float *__restrict__ dweight, float *__restrict__ dbias) {
    wait_for_previous();
    __shared__ float2 stat[VEC * kThreads];   // (m1, m2) of the block's groups
    const int lane = threadIdx.x & 31;
    if ((int)blockIdx.x >= p.N * p.tiles) {
        if (blockIdx.y) return;
        const int wp = threadIdx.x / 32, c = ((int)blockIdx.x - p.N * p.tiles) * 32 + lane;
        float2 v = make_float2(0.f, 0.f);
        if (c < p.C)
            for (int k = wp; k < p.N * p.tiles; k += kThreads / 32) {
                const float2 u = chan[(long long)k * p.C + c];
                v.x += u.x;
                v.y += u.y;
            }
        stat[threadIdx.x] = v;
        __syncthreads();
        if (wp == 0 && c < p.C) {
#pragma unroll
            for (int i = 1; i < kThreads / 32; ++i) {
                v.x += stat[i * 32 + lane].x;
                v.y += stat[i * 32 + lane].y;
            }
            if (dweight) dweight[c] = v.x;
            if (dbias) dbias[c] = v.y;
        }
        return;
    }
    const int tile = blockIdx.x % p.tiles, n = blockIdx.x / p.tiles, z = blockIdx.y;
    const Block<VEC> b(p, z);
    const float inv = 1.f / ((float)p.L * p.D);
    const int lanes = lanes_for(b.g1 - b.g0 + 1), sl = threadIdx.x & (lanes - 1);
    for (int g0 = b.g0 + (int)(threadIdx.x & ~31) / lanes; g0 <= b.g1; g0 += kThreads / lanes) {
        const int g = min(g0 + (int)(threadIdx.x & 31) / lanes, b.g1);
        const int zn = ((g + 1) * p.D - 1) / p.span - first_block(p, g) + 1;
        float s1 = 0.f, s2 = 0.f;
        for (int k = 0; k < zn; ++k) {
            const float2 *at = part + part_at(p, n, g, 0, k);
#pragma unroll 4
            for (int t = sl; t < p.tiles; t += lanes) {
                const float2 v = at[(long long)t * p.ZG];
                s1 += v.x;
                s2 += v.y;
            }
        }
        s1 = lane_sum(s1, lanes);
        s2 = lane_sum(s2, lanes);
        if (sl == 0) stat[g - b.g0] = make_float2(s1 * inv, s2 * inv);
    }
    __syncthreads();
    const int rl = threadIdx.x / p.tpr, cl = threadIdx.x % p.tpr, rows = kThreads / p.tpr;
    const int r0 = tile * p.tile_rows, r1 = r0 + p.rows_of(tile);
    const int cv = z * p.tpr + cl;
    if (rl >= rows || cv >= p.cvecs) return;
    const Affine<VEC> a(p, n, cv, mean, rstd, weight, bias);
    float2 mm[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) mm[e] = stat[(cv * VEC + e) / p.D - b.g0];
    for (int r = r0 + rl; r < r1; r += 2 * rows) {
        float f[2][VEC], dv[2][VEC], gv[2][VEC];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r + i * rows < r1) {
                const long long at = ((long long)n * p.L + r + i * rows) * p.C + (long long)cv * VEC;
                load_vec<T, VEC>(x + at, f[i]);
                load_vec<T, VEC>(dy + at, dv[i]);
                if (GATE) load_vec<T, VEC>(gate + at, gv[i]);
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r + i * rows < r1) {
                float out[VEC], dg;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = (f[i][e] - a.m[e]) * a.rs[e];
                    const float zz = fmaf(h, a.wt[e], a.bs[e]);
                    const float dz = back_act<T, ACT, GATE>(zz, dv[i][e], GATE ? gv[i][e] : 0.f, dg);
                    out[e] = a.rs[e] * (dz * a.wt[e] - mm[e].x - h * mm[e].y);
                }
                store_vec<T, VEC>(dx + ((long long)n * p.L + r + i * rows) * p.C + (long long)cv * VEC, out);
            }
    }
}

// ------------------------------------------------------------------ cluster form

// CTA `rank` of a cluster of K takes rows [rank R, rank R + R) of one sample and one block of
// whole groups: blockIdx.x = (n blocks + block) K + rank.
struct CluGeo {
    int L, C, G, D;
    int blocks, cb;     // channel blocks of a sample, groups of a block
    int K, R;
    float inv_D;        // for the group of a channel of the block: (i + 0.5) / D, exact below 2^20
};
template <typename T>
struct Clu {
    static constexpr int VEC = vec_of<T>();
    int rank, n, g0, ng, c0, w, r0, nr;   // first group, groups, first channel, channels, first row, rows
    int tpr, rl, cl, rows;                // threads of a row; this thread's row lane and vector; row lanes
    bool on;
    float inv_D;
    // the group of a channel of the block
    __device__ __forceinline__ int group(int ch) const { return (int)(((float)ch + 0.5f) * inv_D); }
    __device__ __forceinline__ explicit Clu(const CluGeo &p) {
        inv_D = p.inv_D;
        rank = blockIdx.x % p.K;
        const int b = blockIdx.x / p.K, blk = b % p.blocks;
        n = b / p.blocks;
        g0 = blk * p.cb;
        ng = min(p.cb, p.G - g0);
        c0 = g0 * p.D;
        w = ng * p.D;
        r0 = rank * p.R;
        nr = max(0, min(p.R, p.L - r0));
        tpr = w / VEC;
        rows = kThreads / tpr;
        rl = threadIdx.x / tpr;
        cl = threadIdx.x - rl * tpr;
        on = rl < rows;
    }
    // element offset of this thread's vector in row r of the CTA's rows
    __device__ __forceinline__ long long at(const CluGeo &p, int r) const {
        return ((long long)n * p.L + r0 + r) * p.C + c0 + cl * VEC;
    }
    __device__ __forceinline__ int tile_at(int r) const { return r * w + cl * VEC; }
};
// f(r) over this thread's rows, four at a time
template <int U, typename T, typename F>
__device__ __forceinline__ void clu_rows(const Clu<T> &c, F &&f) {
    if (c.on)
        for (int r = c.rl; r < c.nr; r += U * c.rows) f(r);
}
// Sums over the row lanes of red[rows][w], in place, into red[parts][w] with `parts` = as many
// as keep every thread busy.  Ends with a barrier.
__device__ __forceinline__ int clu_fold_rows(float *red, int rows, int w) {
    const int parts = max(1, min(rows, kThreads / w));
    for (int i0 = 0; i0 < w * parts; i0 += kThreads) {   // more than once only where parts is 1
        const int i = i0 + threadIdx.x, q = parts > 1 ? i / w : 0;
        float v = 0.f;
        if (i < w * parts)
#pragma unroll 4
            for (int r = q; r < rows; r += parts) v += red[r * w + i - q * w];
        __syncthreads();   // what a thread writes another may have read: parts > 1 writes rows that others sum
        if (i < w * parts) red[i] = v;
    }
    __syncthreads();
    return parts;
}
// sum of one group's D channels of red[parts][w], by `lanes` lanes
__device__ __forceinline__ float clu_group_sum(const float *red, int parts, int w, int first, int D, int sl, int lanes) {
    float s = 0.f;
    for (int q = 0; q < parts; ++q)
#pragma unroll 4
        for (int c = sl; c < D; c += lanes) s += red[q * w + first + c];
    return lane_sum(s, lanes);
}

template <typename T, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads) cluster_forward_kernel(CluGeo p, const T *__restrict__ x,
                                                                   const float *__restrict__ weight,
                                                                   const float *__restrict__ bias,
                                                                   const T *__restrict__ gate, T *__restrict__ y,
                                                                   float *__restrict__ mean, float *__restrict__ rstd,
                                                                   float eps) {
    namespace cg = cooperative_groups;
    constexpr int VEC = vec_of<T>(), U = 4;
    using V = Vec<T, VEC>;
    extern __shared__ __align__(16) uint8_t clu_smem[];
    __shared__ float2 local[kThreads], stat[kThreads];   // (mean, m2) of this CTA's rows; (mean, rstd)
    const Clu<T> c(p);
    float *red = reinterpret_cast<float *>(clu_smem);     // [rows][w]
    T *tile = reinterpret_cast<T *>(clu_smem + (size_t)kThreads * VEC * 4);
    cg::cluster_group cluster = cg::this_cluster();

    float acc[VEC] = {};
    clu_rows<U>(c, [&](int r) {
        typename V::Raw raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + u * c.rows < c.nr) raw[u] = ld_raw<typename V::Raw>(x + c.at(p, r + u * c.rows));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + u * c.rows < c.nr) {
                float f[VEC];
                V::open(raw[u], f);
                *reinterpret_cast<typename V::Raw *>(tile + c.tile_at(r + u * c.rows)) = raw[u];
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[e] += f[e];
            }
    });
    const int lanes = lanes_for(c.ng), sl = threadIdx.x & (lanes - 1);
    const float inv_local = c.nr ? 1.f / ((float)c.nr * p.D) : 0.f;
    // each group's sum of `acc` over the CTA
    auto groups = [&](auto &&store) {
        if (c.on)
#pragma unroll
            for (int e = 0; e < VEC; ++e) red[c.tile_at(c.rl) + e] = acc[e];
        __syncthreads();
        const int parts = clu_fold_rows(red, c.rows, c.w);
        for (int q = (int)(threadIdx.x & ~31) / lanes; q < c.ng; q += kThreads / lanes) {
            const int g = min(q + (int)(threadIdx.x & 31) / lanes, c.ng - 1);
            const float v = clu_group_sum(red, parts, c.w, g * p.D, p.D, sl, lanes);
            if (sl == 0) store(g, v);
        }
        __syncthreads();
    };
    groups([&](int g, float v) { local[g].x = v * inv_local; });
    float m[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        m[e] = c.on ? local[c.group(c.cl * VEC + e)].x : 0.f;
        acc[e] = 0.f;
    }
    clu_rows<1>(c, [&](int r) {
        float f[VEC];
        load_vec<T, VEC>(tile + c.tile_at(r), f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = fmaf(f[e] - m[e], f[e] - m[e], acc[e]);
    });
    groups([&](int g, float v) { local[g].y = v; });
    if (p.K > 1) cluster.sync();
    if ((int)threadIdx.x < c.ng) {
        const int g = threadIdx.x;
        const float inv = 1.f / ((float)p.L * p.D);
        float2 v[8];
        float cnt[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = k < p.K ? *cluster.map_shared_rank(&local[g], k) : make_float2(0.f, 0.f);
            cnt[k] = k < p.K ? (float)max(0, min(p.R, p.L - k * p.R)) * p.D : 0.f;
        }
        float mu = 0.f, q = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) mu = fmaf(cnt[k], v[k].x, mu);
        mu *= inv;
#pragma unroll
        for (int k = 0; k < 8; ++k) q += fmaf(cnt[k] * (v[k].x - mu), v[k].x - mu, v[k].y);
        const float rs = rsqrtf(q * inv + eps);
        stat[g] = make_float2(mu, rs);
        if (c.rank == 0) {
            mean[(long long)c.n * p.G + c.g0 + g] = mu;
            rstd[(long long)c.n * p.G + c.g0 + g] = rs;
        }
    }
    if (p.K > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");   // nobody leaves while its sums are read
    __syncthreads();
    float sc[VEC], o[VEC];   // z = (x - m) sc + o
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int ch = c.cl * VEC + e;
        const float2 v = c.on ? stat[c.group(ch)] : make_float2(0.f, 0.f);
        m[e] = v.x;
        sc[e] = v.y * (weight && c.on ? weight[c.c0 + ch] : 1.f);
        o[e] = bias && c.on ? bias[c.c0 + ch] : 0.f;
    }
    clu_rows<U>(c, [&](int r) {
        typename V::Raw gr[U];
        if (GATE)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * c.rows < c.nr) gr[u] = ld_raw<typename V::Raw>(gate + c.at(p, r + u * c.rows));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + u * c.rows < c.nr) {
                float f[VEC], gv[VEC], out[VEC];
                load_vec<T, VEC>(tile + c.tile_at(r + u * c.rows), f);
                if (GATE) V::open(gr[u], gv);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float z = fmaf(f[e] - m[e], sc[e], o[e]);
                    out[e] = GATE ? z * act<T, ACT>(gv[e]) : act<T, ACT>(z);
                }
                st_raw(y + c.at(p, r + u * c.rows), V::close(out));
            }
    });
    if (p.K > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// part: [N][2][C] sums of dz xhat and dz of each sample (dweight and dbias themselves when N = 1)
template <typename T, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads) cluster_backward_kernel(
    CluGeo p, const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
    const float *__restrict__ rstd, const float *__restrict__ weight, const float *__restrict__ bias,
    const T *__restrict__ gate, T *__restrict__ dx, T *__restrict__ dgate, float *__restrict__ part_w,
    float *__restrict__ part_b, long long part_stride) {
    namespace cg = cooperative_groups;
    constexpr int VEC = vec_of<T>(), U = 4, NT = GATE ? 3 : 2;
    using V = Vec<T, VEC>;
    let_next_start();
    extern __shared__ __align__(16) uint8_t clu_smem[];
    __shared__ float2 stat[kThreads];   // (m1, m2) of the groups
    const Clu<T> c(p);
    // [rows][w] sums of dz xhat, then of dz; the first w of each become the CTA's channel sums, which the
    // other CTAs read; then this thread block's totals
    float *red_w = reinterpret_cast<float *>(clu_smem), *red_b = red_w + kThreads * VEC, *tot_w = red_b + kThreads * VEC,
          *tot_b = tot_w + kThreads * VEC;
    T *tile = reinterpret_cast<T *>(tot_b + kThreads * VEC);
    const int plane = p.R * c.w;        // elements of one tensor's tile
    cg::cluster_group cluster = cg::this_cluster();
    float m[VEC], rs[VEC], wt[VEC], bs[VEC], dw[VEC] = {}, db[VEC] = {};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int in = c.on ? c.cl * VEC + e : 0, ch = c.c0 + in;
        const long long i = (long long)c.n * p.G + c.g0 + c.group(in);
        m[e] = mean[i];
        rs[e] = rstd[i];
        wt[e] = weight ? weight[ch] : 1.f;
        bs[e] = bias ? bias[ch] : 0.f;
    }
    clu_rows<U>(c, [&](int r) {
        typename V::Raw raw[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + u * c.rows < c.nr) {
                const long long at = c.at(p, r + u * c.rows);
                raw[u][0] = ld_raw<typename V::Raw>(x + at);
                raw[u][1] = ld_raw<typename V::Raw>(dy + at);
                if (GATE) raw[u][NT - 1] = ld_raw<typename V::Raw>(gate + at);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + u * c.rows < c.nr) {
                float f[VEC], dv[VEC], gv[VEC], dg[VEC];
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    *reinterpret_cast<typename V::Raw *>(tile + k * plane + c.tile_at(r + u * c.rows)) = raw[u][k];
                V::open(raw[u][0], f);
                V::open(raw[u][1], dv);
                if (GATE) V::open(raw[u][NT - 1], gv);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = (f[e] - m[e]) * rs[e];
                    const float z = fmaf(h, wt[e], bs[e]);
                    const float dz = back_act<T, ACT, GATE>(z, dv[e], GATE ? gv[e] : 0.f, dg[e]);
                    dw[e] = fmaf(dz, h, dw[e]);
                    db[e] += dz;
                }
                if (GATE) st_raw(dgate + c.at(p, r + u * c.rows), V::close(dg));
            }
    });
    if (c.on)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            red_w[c.tile_at(c.rl) + e] = dw[e];
            red_b[c.tile_at(c.rl) + e] = db[e];
        }
    __syncthreads();
    const int parts = clu_fold_rows(red_w, c.rows, c.w);
    clu_fold_rows(red_b, c.rows, c.w);
    if (parts > 1) {
        for (int i = threadIdx.x; i < c.w; i += kThreads) {   // (w < kThreads here)
            float a = red_w[i], b = red_b[i];
            for (int k = 1; k < parts; ++k) {
                a += red_w[k * c.w + i];
                b += red_b[k * c.w + i];
            }
            red_w[i] = a;
            red_b[i] = b;
        }
    }
    if (p.K > 1) cluster.sync();
    else __syncthreads();
    for (int i = threadIdx.x; i < c.w; i += kThreads) {
        float va[8], vb[8], a = 0.f, b = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            va[k] = k < p.K ? *cluster.map_shared_rank(red_w + i, k) : 0.f;
            vb[k] = k < p.K ? *cluster.map_shared_rank(red_b + i, k) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            a += va[k];
            b += vb[k];
        }
        if (c.rank == 0) {
            if (part_w) part_w[c.n * part_stride + c.c0 + i] = a;
            if (part_b) part_b[c.n * part_stride + c.c0 + i] = b;
        }
        const float wc = weight ? weight[c.c0 + i] : 1.f;
        tot_w[i] = wc * a;
        tot_b[i] = wc * b;
    }
    if (p.K > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");   // nobody leaves while its sums are read
    __syncthreads();
    const int lanes = lanes_for(c.ng), sl = threadIdx.x & (lanes - 1);
    const float inv = 1.f / ((float)p.L * p.D);
    for (int q = (int)(threadIdx.x & ~31) / lanes; q < c.ng; q += kThreads / lanes) {
        const int g = min(q + (int)(threadIdx.x & 31) / lanes, c.ng - 1);
        const float s1 = clu_group_sum(tot_b, 1, c.w, g * p.D, p.D, sl, lanes);
        const float s2 = clu_group_sum(tot_w, 1, c.w, g * p.D, p.D, sl, lanes);
        if (sl == 0) stat[g] = make_float2(s1 * inv, s2 * inv);
    }
    __syncthreads();
    float2 mm[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) mm[e] = c.on ? stat[c.group(c.cl * VEC + e)] : make_float2(0.f, 0.f);
    clu_rows<1>(c, [&](int r) {
        float f[VEC], dv[VEC], gv[VEC], out[VEC], dg;
        load_vec<T, VEC>(tile + c.tile_at(r), f);
        load_vec<T, VEC>(tile + plane + c.tile_at(r), dv);
        if (GATE) load_vec<T, VEC>(tile + 2 * plane + c.tile_at(r), gv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float h = (f[e] - m[e]) * rs[e];
            const float z = fmaf(h, wt[e], bs[e]);
            const float dz = back_act<T, ACT, GATE>(z, dv[e], GATE ? gv[e] : 0.f, dg);
            out[e] = rs[e] * (dz * wt[e] - mm[e].x - h * mm[e].y);
        }
        st_raw(dx + c.at(p, r), V::close(out));
    });
    if (p.K > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// dweight (blockIdx.y 0) or dbias (1) from the rows form's partial sums [reps][2][C]: 32
// channels a CTA, 32 warps over the partial sums.
__global__ void __launch_bounds__(1024) rows_back_join_kernel(const float *__restrict__ part, int reps, long long C,
                                                              float *__restrict__ dweight, float *__restrict__ dbias) {
    wait_for_previous();
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, wp = threadIdx.x / 32;
    const long long c = (long long)blockIdx.x * 32 + lane;
    float *dst = blockIdx.y ? dbias : dweight;
    if (!dst) return;
    part += blockIdx.y * C;
    float v = 0.f;
    if (c < C) {
#pragma unroll 4
        for (int k = wp; k < reps; k += 32) v += part[k * 2 * C + c];
    }
    s[wp][lane] = v;
    __syncthreads();
    // warp wp sums channel wp's 32 entries, in the same order every time
    v = lane_sum(s[lane][wp], 32);
    if (lane == 0 && (long long)blockIdx.x * 32 + wp < C) dst[(long long)blockIdx.x * 32 + wp] = v;
}

}  // namespace norm
}  // namespace kda

// ------------------------------------------------------------------ host side

namespace kda {
namespace norm {

constexpr int kSMs = 148;

struct Plan {
    bool rows;          // rows form
    bool cluster;       // cluster form
    CluGeo c;
    size_t smem;        // of a CTA of the cluster form
    RowsGeo r;
    int nv, row_blocks;
    PosGeo p;
    bool vec;           // positions form: 16-byte vectors
    size_t ws;          // workspace bytes
};

inline long long gcd_of(long long a, long long b) { return b ? gcd_of(b, a % b) : a; }

// Cluster form: blocks of the fewest groups that are whole vectors and at least 64 bytes of a
// row (a half-used sector costs more than it saves below that), and the fewest CTAs that leave
// room for several an SM and fill the GPU.  Beyond eight CTAs' shared memory the positions form
// takes over, and for gradients above kClusterGrad elements, where a CTA's chain of barriers
// costs more than the second read.  Measured, us, cluster | positions, bf16:
//   forward   3 x 4096 x 320, 32 groups 16 | 23;  8 x 512 x 512, 8 groups 12 | 16;  4 x 64 x 72 10 | 18
//   gradients 3 x 4096 x 320 27 | 22;  8 x 512 x 512 22 | 16;  2 x 1021 x 640 fp32 14 | 16;  1 x 2 x 64 8 | 10
// Forward the cluster wins or is equal in all of 22 sizes of 13 thousand to 4 million elements.  The gradients' border lies
// between 1.2 and 4 million and no count of elements draws it exactly.  Positions are taken at 3 x 2048 x 320 14.5 | 16.4,
// 64 x 128 x 320 18.5 | 20.5, 512 x 16 x 256 20.5 | 22.6, fp32 4 x 1024 x 512 14.4 | 16.4 and 1 x 4096 x 512 12.3 | 18.5, and
// the cluster at fp32 with a gate 2 x 1021 x 640 18.5 | 16.5; in the 16 other sizes measured it takes the faster one or one within 4 %.
constexpr size_t kClusterWant = 56 * 1024, kClusterSmem = 200 * 1024;
constexpr long long kClusterGrad = 3 << 19;
inline bool cluster_plan(long long N, int L, int C, int G, int esize, bool gated, bool backward, Plan &s) {
    const int vw = 16 / esize, D = C / G, unit = vw / (int)gcd_of(D, vw);
    if (C % vw || (backward && N * L * C > kClusterGrad)) return false;
    int cb = unit;
    while (cb < G && (long long)cb * D * esize < 64) cb += unit;
    // wider while there are CTAs enough without it
    const int tensors = backward ? (gated ? 3 : 2) : 1;
    while (cb < G && N * ((G + 2 * cb - 1) / (2 * cb)) >= 2 * kSMs && (long long)2 * cb * D <= kThreads * vw &&
           (size_t)L * 2 * cb * D * esize * tensors <= kClusterWant)
        cb *= 2;
    cb = std::min(cb, G);
    const long long vecs = (long long)cb * D / vw;
    if (vecs > kThreads || cb > kThreads) return false;
    const int blocks = (G + cb - 1) / cb, rows = kThreads / (int)vecs;
    const size_t fixed = (size_t)kThreads * vw * 4 * (backward ? 4 : 1);
    for (int K = 1; K <= 8; K *= 2) {
        const int R = (L + K - 1) / K;
        const size_t smem = fixed + (size_t)R * cb * D * esize * tensors;
        if (K < 8 && (smem > kClusterWant || (N * blocks * K < kSMs && R > rows))) continue;
        if (smem > kClusterSmem) return false;
        s.cluster = true;
        s.c = CluGeo{L, C, G, D, blocks, cb, K, R, 1.f / D};
        s.smem = smem;
        s.ws = backward && N > 1 ? (size_t)N * 2 * C * sizeof(float) : 0;
        return N * blocks * K < (1ll << 31);
    }
    return false;
}

// Rows form up to four vectors a lane (D <= 1024 bf16, 512 fp32); beyond that, or with
// several positions, the statistics span CTAs.
inline Plan plan_of(long long N, int L, int C, int G, int esize, bool gated, bool backward) {
    Plan s{};
    const int vw = 16 / esize, D = C / G;
    if (L == 1 && D % vw == 0 && D / vw <= 128) {
        s.rows = true;
        const int vecs = D / vw;
        int lanes = 1;
        while (lanes < vecs && lanes < 32) lanes *= 2;
        const int nv = (vecs + lanes - 1) / lanes;
        s.nv = nv <= 2 ? nv : 4;
        const long long rows = N * G, per = kThreads / lanes;
        const long long unit = G / gcd_of(G, per);   // blocks whose lane groups are a multiple of G
        const long long want = std::min<long long>((rows + per - 1) / per,
                                                   (long long)kSMs * rows_ctas(s.nv, backward));
        s.row_blocks = (int)std::max(want / unit, 1ll) * (int)unit;   // whole units, no more CTAs than fit
        s.r = RowsGeo{rows, G, D, lanes, (int)(s.row_blocks * per)};
        s.ws = backward ? (size_t)(s.r.step / G) * 2 * C * sizeof(float) : 0;
        return s;
    }
    if (cluster_plan(N, L, C, G, esize, gated, backward, s)) return s;
    s.cluster = false;
    s.ws = 0;
    s.vec = C % vw == 0;
    PosGeo &p = s.p;
    p.N = (int)N; p.L = L; p.C = C; p.G = G; p.D = D;
    p.cvecs = s.vec ? C / vw : C;
    p.tpr = std::min(p.cvecs, kThreads);
    p.Z = (p.cvecs + p.tpr - 1) / p.tpr;
    p.span = p.tpr * (s.vec ? vw : 1);
    p.ZG = std::min(p.Z, (D + p.span - 2) / p.span + 1);
    const int rows = kThreads / p.tpr;                       // rows a CTA holds at a time
    const long long want = std::max<long long>(1, 2 * kSMs / (N * p.Z));   // tiles of a sample: two CTAs per SM
    const long long tr = std::max<long long>((L + want - 1) / want, (long long)8 * rows);
    p.tile_rows = (int)std::min<long long>(tr, L);
    p.tiles = (L + p.tile_rows - 1) / p.tile_rows;
    const size_t group = (size_t)N * G * p.tiles * p.ZG * sizeof(float2);
    s.ws = group + (backward ? (size_t)N * p.tiles * C * sizeof(float2) : 0);
    return s;
}

struct Args {
    const void *dy, *x, *gate;
    const float *weight, *bias;
    void *y, *dgate;          // y or dx
    float *mean, *rstd;       // backward: read only
    float *dweight, *dbias;
    float eps;
    void *ws;
    long long N;
};

// Heads of 64 and 128 channels have kernels of their own widths.
#define KDA_ROWS_CASES                                        \
    if (s.nv == 1) {                                          \
        const int exact = s.r.D == s.r.lanes * VW ? s.r.lanes : 0; \
        if (exact == 8) KDA_ROWS(1, 8);                       \
        else if (exact == 16) KDA_ROWS(1, 16);                \
        else if (exact == 32) KDA_ROWS(1, 32);                \
        else KDA_ROWS(1, 0);                                  \
    } else if (s.nv == 2) {                                   \
        KDA_ROWS(2, 0);                                       \
    } else {                                                  \
        KDA_ROWS(4, 0);                                       \
    }

template <typename... Params, typename... A>
cudaError_t launch_cluster(void (*kern)(Params...), const Plan &s, long long N, cudaStream_t st, A &&...args) {
    // one limit for every plan: another host thread may be between its own call of this and its launch
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kClusterSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = s.c.K;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(N * s.c.blocks * s.c.K));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

template <typename T, int ACT, bool GATE>
cudaError_t launch_forward(const Plan &s, const Args &a, cudaStream_t st) {
    constexpr int VW = vec_of<T>();
    const T *x = (const T *)a.x, *gate = (const T *)a.gate;
    T *y = (T *)a.y;
    if (s.rows) {
#define KDA_ROWS(NV, LANES)                                                                                     \
    rows_forward_kernel<T, NV, LANES, ACT, GATE><<<s.row_blocks, kThreads, 0, st>>>(s.r, x, a.weight, a.bias, gate, y, \
                                                                                    a.mean, a.rstd, a.eps)
        KDA_ROWS_CASES
#undef KDA_ROWS
        return cudaGetLastError();
    }
    if (s.cluster)
        return launch_cluster(cluster_forward_kernel<T, ACT, GATE>, s, a.N, st, s.c, x, a.weight, a.bias, gate, y, a.mean,
                              a.rstd, a.eps);
    const dim3 grid((unsigned)((long long)s.p.N * s.p.tiles), s.p.Z);
    float2 *part = (float2 *)a.ws;
    auto run = [&](auto moments, auto apply) {
        moments<<<grid, kThreads, 0, st>>>(s.p, x, part);
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess ? e
                                : launch_after(apply, grid, kThreads, 0, st, s.p, x, a.weight, a.bias, gate, y, part,
                                               a.mean, a.rstd, a.eps);
    };
    if (s.vec) return run(pos_moments_kernel<T, VW>, pos_apply_kernel<T, VW, ACT, GATE>);
    return run(pos_moments_kernel<T, 1>, pos_apply_kernel<T, 1, ACT, GATE>);
}

template <typename T, int ACT, bool GATE>
cudaError_t launch_backward(const Plan &s, const Args &a, cudaStream_t st) {
    constexpr int VW = vec_of<T>();
    const T *dy = (const T *)a.dy, *x = (const T *)a.x, *gate = (const T *)a.gate;
    T *dx = (T *)a.y, *dgate = (T *)a.dgate;
    if (s.rows) {
        float *part = (float *)a.ws;
        const long long C = (long long)s.r.G * s.r.D;
#define KDA_ROWS(NV, LANES)                                                                                     \
    rows_backward_kernel<T, NV, LANES, ACT, GATE><<<s.row_blocks, kThreads, 0, st>>>(s.r, dy, x, a.mean, a.rstd, a.weight, \
                                                                                     a.bias, gate, dx, dgate, part)
        KDA_ROWS_CASES
#undef KDA_ROWS
        if (a.dweight || a.dbias)
            return launch_after(rows_back_join_kernel, dim3((unsigned)((C + 31) / 32), 2), 1024, 0, st, part,
                                s.r.step / s.r.G, C, a.dweight, a.dbias);
        return cudaGetLastError();
    }
    if (s.cluster) {
        const bool one = a.N == 1, join = !one && (a.dweight || a.dbias);
        float *part = (float *)a.ws;
        const cudaError_t e = launch_cluster(cluster_backward_kernel<T, ACT, GATE>, s, a.N, st, s.c, dy, x, a.mean, a.rstd,
                                             a.weight, a.bias, gate, dx, dgate, one ? a.dweight : join ? part : nullptr,
                                             one ? a.dbias : join ? part + s.c.C : nullptr, 2ll * s.c.C);
        if (e != cudaSuccess || !join) return e;
        return launch_after(rows_back_join_kernel, dim3((unsigned)((s.c.C + 31) / 32), 2), 1024, 0, st, part, (int)a.N,
                            (long long)s.c.C, a.dweight, a.dbias);
    }
    const long long tiles = (long long)s.p.N * s.p.tiles;
    const dim3 grid((unsigned)tiles, s.p.Z);
    const unsigned join = a.dweight || a.dbias ? (s.p.C + 31) / 32 : 0;
    float2 *part = (float2 *)a.ws, *chan = part + (size_t)s.p.N * s.p.G * s.p.tiles * s.p.ZG;
    auto run = [&](auto sums, auto apply) {
        sums<<<grid, kThreads, 0, st>>>(s.p, dy, x, a.mean, a.rstd, a.weight, a.bias, gate, dgate, chan, part);
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess ? e
                                : launch_after(apply, dim3(grid.x + join, grid.y), kThreads, 0, st, s.p, dy, x, a.mean,
                                               a.rstd, a.weight, a.bias, gate, dx, chan, part, a.dweight, a.dbias);
    };
    if (s.vec) return run(pos_back_sums_kernel<T, VW, ACT, GATE>, pos_back_apply_kernel<T, VW, ACT, GATE>);
    return run(pos_back_sums_kernel<T, 1, ACT, GATE>, pos_back_apply_kernel<T, 1, ACT, GATE>);
}

template <typename T>
cudaError_t launch(const Plan &s, const Args &a, int act, bool backward, cudaStream_t st) {
#define KDA_NORM(ACT)                                                                                       \
    return backward ? (a.gate ? launch_backward<T, ACT, true>(s, a, st) : launch_backward<T, ACT, false>(s, a, st)) \
                    : (a.gate ? launch_forward<T, ACT, true>(s, a, st) : launch_forward<T, ACT, false>(s, a, st))
    if (act == KDA_ACT_NONE) KDA_NORM(KDA_ACT_NONE);
    if (act == KDA_ACT_SILU) KDA_NORM(KDA_ACT_SILU);
    KDA_NORM(KDA_ACT_SIGMOID);
#undef KDA_NORM
}

}  // namespace norm
}  // namespace kda

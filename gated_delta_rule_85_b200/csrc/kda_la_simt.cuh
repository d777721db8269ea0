// Linear attention with a decay for each head on CUDA cores: the walk and the first
// pass in fp32, 64 tokens a chunk, for any supported dtype and head size.
//
// One 256-thread CTA takes one span.  The state lives in registers (thread (ty, tx)
// of a 16 x 16 grid holds DAB/16 rows x DC/16 columns) and is put in shared memory
// once a chunk for the product with the a rows.
//
// Bound by latency with one CTA of 8 warps an SM and by its shared-memory reads (a 16-byte read is four
// wavefronts, whoever shares it; 40 % of the cycles): 2 x 1003 tokens x 8 heads of 64 x 128 take 65 us, of which the
// walk 42 in spans of one and two chunks (64 of 128 columns a CTA, two CTAs an SM: 50; 512 threads of two token rows:
// 55); its gradients take 164.
#pragma once

#include "kda_la.cuh"
#include "kda_launch.cuh"

namespace kda {
namespace la {

constexpr int kSimtC = 64;

// One walk: out = linear attention of rows a on rows b, c (see kda_la.cuh).
struct Walk {
    const void *a, *b, *c;
    void *out;
    Carry y;
    bool transposed;    // the states it reads are [DC][DAB]; it writes none then
};

template <int DAB, int DC>
struct SimtSmem {
    static constexpr int SA = DAB + 4, SP = kSimtC + 4;   // row strides in floats: 16-byte rows, no bank conflicts
    static constexpr int A = 0;                           // [64][SA]
    static constexpr int B = A + kSimtC * SA;             // [64][SA]
    static constexpr int CT = B + kSimtC * SA;            // [64][DC]
    static constexpr int X = CT + kSimtC * DC;            // [DAB][DC]
    static constexpr int P = X + DAB * DC;                // [64][SP]
    static constexpr int PW = P + kSimtC * SP;            // [65] powers of g
    static constexpr size_t bytes = (PW + 68) * sizeof(float);
};

// rows [t, t + len) of one head -> shared memory as fp32, zeros behind them
template <int D, typename Tin>
__device__ __forceinline__ void simt_load(float *dst, int stride, const Tin *src, long long t, int len, int H, int h) {
    for (int i = threadIdx.x; i < kSimtC * (D / 4); i += 256) {
        const int r = i / (D / 4), x = (i % (D / 4)) * 4;
        const float4 v = r < len ? load4(src + ((t + r) * H + h) * D + x) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(dst + r * stride + x) = v;
    }
}

// WALK: the outputs, and the final states; else the first pass: sums of the parts that
// go on behind their span.  DIR: 1 forwards, -1 backwards in time.
template <int DAB, int DC, typename Tin, int DIR, bool WALK>
__global__ void __launch_bounds__(256) la_simt_kernel(Geo g, Walk wk, const float *__restrict__ log_decay,
                                                      const int32_t *__restrict__ slots, int num_slots) {
    using L = SimtSmem<DAB, DC>;
    constexpr int RM = DAB / 16, CG = DC / 64;   // state rows of a thread; its columns: 4 tx + 64 j
    let_next_start();
    wait_for_previous();
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int w = blockIdx.x;
    const long long lo = g.lo(w), hi = g.hi(w);
    const long long E = DAB * DC;
    const Carry &y = wk.y;

    float S[RM][CG * 4];
    int head = -1;
    float lg = 0.f;
    Cursor<kSimtC> cur;
    cur.valid = false;
    bool fresh = true;    // the next item is the first valid one of the span
    for (long long i = 0; i < hi - lo; ++i) {
        const long long u = DIR > 0 ? lo + i : hi - 1 - i;
        if (i == 0) cur.seek(g, u);
        else cur.template step<DIR>(g, u);
        if (!cur.valid) continue;
        const bool begins = cur.c == (DIR > 0 ? 0 : cur.nck - 1);
        const bool ends = cur.c == (DIR > 0 ? cur.nck - 1 : 0);
        // does the sequence's last item in walking order lie in this span?
        const long long u_end = DIR > 0 ? u + (cur.nck - 1 - cur.c) : u - cur.c;
        const bool whole_tail = u_end >= lo && u_end < hi;
        const bool from_before = fresh && !begins;
        const bool first = fresh || begins;
        fresh = false;
        if (!WALK && whole_tail) continue;   // nothing goes on behind the span: no sum is needed
        const int len = cur.len();
        const long long t = cur.tok();
        const int h = cur.h;
        __syncthreads();   // the chunk before is done with shared memory
        if (h != head) {
            head = h;
            lg = rate_of(log_decay, h);
            if (tid <= kSimtC) sm[L::PW + tid] = (float)exp((double)lg * tid);
        }
        if (first) {
            const int row = state_row(slots, num_slots, cur.n);
            const float *src = nullptr;
            if (from_before) {
                if (WALK) src = y.start + w * E;
            } else if (WALK) {
                if (y.s0_copy && !whole_tail) src = y.s0_copy + ((long long)cur.n * g.H + h) * E;
                else if (y.s0 && row >= 0) src = y.s0 + ((long long)row * g.H + h) * E;
            }
#pragma unroll
            for (int r = 0; r < RM; ++r)
#pragma unroll
                for (int j = 0; j < CG * 4; ++j) {
                    const int rr = ty * RM + r, cc = tx * 4 + (j >> 2) * 64 + (j & 3);
                    S[r][j] = src ? (wk.transposed ? src[cc * DAB + rr] : src[rr * DC + cc]) : 0.f;
                }
        }
        if (WALK) simt_load<DAB>(sm + L::A, L::SA, (const Tin *)wk.a, t, len, g.H, h);
        simt_load<DAB>(sm + L::B, L::SA, (const Tin *)wk.b, t, len, g.H, h);
        simt_load<DC>(sm + L::CT, DC, (const Tin *)wk.c, t, len, g.H, h);
        if (WALK) {
#pragma unroll
            for (int r = 0; r < RM; ++r)
#pragma unroll
                for (int j = 0; j < CG; ++j)
                    *reinterpret_cast<float4 *>(sm + L::X + (ty * RM + r) * DC + tx * 4 + j * 64) =
                        make_float4(S[r][4 * j], S[r][4 * j + 1], S[r][4 * j + 2], S[r][4 * j + 3]);
        }
        __syncthreads();
        if (WALK) {
            // scores of rows 4 ty + i, columns tx + 16 j
            float p[4][4] = {};
#pragma unroll 4
            for (int d = 0; d < DAB; d += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[k] = *reinterpret_cast<const float4 *>(sm + L::A + (ty * 4 + k) * L::SA + d);
                    b[k] = *reinterpret_cast<const float4 *>(sm + L::B + (tx + 16 * k) * L::SA + d);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        p[r][j] = fmaf(a[r].x, b[j].x, fmaf(a[r].y, b[j].y,
                                  fmaf(a[r].z, b[j].z, fmaf(a[r].w, b[j].w, p[r][j]))));
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = (ty * 4 + r - tx - 16 * j) * DIR;
                    sm[L::P + (ty * 4 + r) * L::SP + tx + 16 * j] = d >= 0 ? p[r][j] * sm[L::PW + d] : 0.f;
                }
            // out rows 4 ty + r, columns 4 tx + 64 j
            float o[4][CG * 4] = {};
#pragma unroll 2
            for (int d = 0; d < DAB; d += 4) {
                float4 a[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    a[r] = *reinterpret_cast<const float4 *>(sm + L::A + (ty * 4 + r) * L::SA + d);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < CG; ++j) {
                        const float4 x = *reinterpret_cast<const float4 *>(sm + L::X + (d + k) * DC + tx * 4 + j * 64);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float ak = k == 0 ? a[r].x : k == 1 ? a[r].y : k == 2 ? a[r].z : a[r].w;
                            o[r][4 * j] = fmaf(ak, x.x, o[r][4 * j]);
                            o[r][4 * j + 1] = fmaf(ak, x.y, o[r][4 * j + 1]);
                            o[r][4 * j + 2] = fmaf(ak, x.z, o[r][4 * j + 2]);
                            o[r][4 * j + 3] = fmaf(ak, x.w, o[r][4 * j + 3]);
                        }
                    }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i2 = ty * 4 + r;
                const float up = sm[L::PW + (DIR > 0 ? i2 + 1 : max(len - 1 - i2, 0))];
#pragma unroll
                for (int j = 0; j < CG * 4; ++j) o[r][j] *= up;
            }
            __syncthreads();   // P is complete
#pragma unroll 2
            for (int d = 0; d < kSimtC; d += 4) {
                float4 a[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    a[r] = *reinterpret_cast<const float4 *>(sm + L::P + (ty * 4 + r) * L::SP + d);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < CG; ++j) {
                        const float4 x = *reinterpret_cast<const float4 *>(sm + L::CT + (d + k) * DC + tx * 4 + j * 64);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float ak = k == 0 ? a[r].x : k == 1 ? a[r].y : k == 2 ? a[r].z : a[r].w;
                            o[r][4 * j] = fmaf(ak, x.x, o[r][4 * j]);
                            o[r][4 * j + 1] = fmaf(ak, x.y, o[r][4 * j + 1]);
                            o[r][4 * j + 2] = fmaf(ak, x.z, o[r][4 * j + 2]);
                            o[r][4 * j + 3] = fmaf(ak, x.w, o[r][4 * j + 3]);
                        }
                    }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (ty * 4 + r < len)
#pragma unroll
                    for (int j = 0; j < CG; ++j)
                        store4((Tin *)wk.out + ((t + ty * 4 + r) * g.H + h) * DC + tx * 4 + j * 64,
                               make_float4(o[r][4 * j], o[r][4 * j + 1], o[r][4 * j + 2], o[r][4 * j + 3]));
        }
        // S <- g^len S + sum_j weight_j b_j c_j^T; rows behind len are zeros
        const float2 dec = decay2(lg, len);
#pragma unroll
        for (int r = 0; r < RM; ++r)
#pragma unroll
            for (int j = 0; j < CG * 4; ++j) S[r][j] = fmaf(dec.x, S[r][j], dec.y * S[r][j]);
#pragma unroll 2
        for (int j = 0; j < len; ++j) {
            const float wt = sm[L::PW + (DIR > 0 ? len - 1 - j : j + 1)];
            float4 cc[CG];
#pragma unroll
            for (int x = 0; x < CG; ++x) {
                cc[x] = *reinterpret_cast<const float4 *>(sm + L::CT + j * DC + tx * 4 + x * 64);
                cc[x].x *= wt; cc[x].y *= wt; cc[x].z *= wt; cc[x].w *= wt;
            }
#pragma unroll
            for (int r = 0; r < RM; r += 4) {
                const float4 b = *reinterpret_cast<const float4 *>(sm + L::B + j * L::SA + ty * RM + r);
#pragma unroll
                for (int x = 0; x < CG; ++x)
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr) {
                        const float bk = rr == 0 ? b.x : rr == 1 ? b.y : rr == 2 ? b.z : b.w;
                        S[r + rr][4 * x] = fmaf(bk, cc[x].x, S[r + rr][4 * x]);
                        S[r + rr][4 * x + 1] = fmaf(bk, cc[x].y, S[r + rr][4 * x + 1]);
                        S[r + rr][4 * x + 2] = fmaf(bk, cc[x].z, S[r + rr][4 * x + 2]);
                        S[r + rr][4 * x + 3] = fmaf(bk, cc[x].w, S[r + rr][4 * x + 3]);
                    }
            }
        }
        // the part is over: its state or its sum
        float *dst = nullptr;
        if (WALK) {
            if (ends && y.last) {
                const int row = state_row(slots, num_slots, cur.n);
                if (row >= 0) dst = y.last + ((long long)row * g.H + h) * E;
            }
        } else if (i == hi - lo - 1) {
            // through: the sequence came from the span before
            const long long u_beg = DIR > 0 ? u - cur.c : u + (cur.nck - 1 - cur.c);
            dst = (u_beg >= lo && u_beg < hi ? y.sum_out : y.sum_in) + w * E;
        }
        if (dst) {
#pragma unroll
            for (int r = 0; r < RM; ++r)
#pragma unroll
                for (int j = 0; j < CG * 4; ++j) {
                    const int rr = ty * RM + r, cc = tx * 4 + (j >> 2) * 64 + (j & 3);
                    dst[rr * DC + cc] = S[r][j];
                }
        }
    }
}

}  // namespace la
}  // namespace kda

// ------------------------------------------------------------------ host side

namespace kda {
namespace la {

// Sizes of one call, from the host's arguments.
struct Call {
    const int32_t *cu, *slots;
    int B, T, H, N, num_slots;
    const float *log_decay;
    cudaStream_t st;
};

// Cut spans give every SM the same share, but cost a first pass over k and v, a join and two
// more launches.  A dense batch is cut only where whole sequences take longer, by a model in
// chunks of one walk: `walks` walks and `sums` first passes, side by side in one launch or one
// after the other.  Measured on the way to its constants, us, cut | whole:
//   bf16 forward   2 x 300 x 32 heads of 128 39 | 25;  8 x 2048 x 32 222 | 165;  4 x 1000 x 8 37 | 47
//   bf16 gradients 4 x 1000 x 8 heads of 128 75 | 48;  8 x 2048 x 32 532 | 402;  1 x 1500 x 4 29 | 63
//   fp32 forward   8 x 500 x 16 heads of 64 164 | 91;  1 x 200 x 8 44 | 94
// and behind them, where the rule takes the slower side: gradients of 2 x 2000 x 16 heads of 64 x 128 92 | 121 (whole;
// two launches of walks there, the model counts one) and of 4 x 2048 x 16 heads of 128 172 | 150 (cut); fp32 2 x 500 x
// 40 heads of 64 130 | 100 forward, 370 | 317 gradients (cut).  In 38 other measurements it takes the faster one, heads of
// 64, of 128 and mixed in either type.
template <int C>
Geo geo_of(const Call &c, int walks, int sums, bool side_by_side) {
    Geo g{c.cu, c.T, c.N, c.H, 0, 0, 0, 0, 1};
    const int nck = (c.T + C - 1) / C;
    g.nslots = (int)(c.cu ? (long long)c.T / C + c.N : (long long)c.N * nck);
    if (!c.cu) {
        auto rounds = [](long long ctas) { return (float)((ctas + kSMs - 1) / kSMs); };
        const float sum = C == kSimtC ? 0.45f : 0.63f, fixed = C == kSimtC ? 0.5f : 1.9f;
        const long long seqs = (long long)c.H * c.N, ctas = std::min<long long>(g.items(), kSMs);
        const float part = rounds(g.items());   // the longest cut span
        float cut = fixed, whole;
        if (side_by_side) {
            cut += (sum * rounds(sums * ctas) + rounds(walks * ctas)) * part;
            whole = seqs <= kSMs ? rounds(walks * seqs)
                                 : std::min(walks * rounds(seqs), (float)(walks * seqs) / kSMs + 1.f);
        } else {
            cut += (sum * sums + walks) * part;
            whole = walks * rounds(seqs);
        }
        if (whole * nck <= cut) g.unit = nck;
    }
    const long long units = g.items() / g.unit;
    g.W = (int)std::min<long long>(units, kSMs);
    g.per = units / g.W;
    g.rem = (int)(units % g.W);
    return g;
}

// Does a span boundary fall inside a sequence?  Packed lengths are on the device: any of
// more than one chunk may be cut.
template <int C>
bool cuts(const Geo &g) {
    if (g.T <= C || g.unit > 1) return false;
    if (g.cu) return true;
    const int per = (g.T + C - 1) / C;
    for (int w = 1; w < g.W; ++w)
        if (g.lo(w) % per) return true;
    return false;
}

// Workspace of one set of carried states.
inline size_t carry_bytes(int W, int dk, int dv) { return (size_t)3 * W * dk * dv * sizeof(float); }
inline Carry carry_at(float *ws, int W, int E) {
    Carry y{};
    y.sum_in = ws;
    y.sum_out = ws + (size_t)W * E;
    y.start = ws + (size_t)2 * W * E;
    return y;
}

// One or two sets of carried states (directions `dirs`); the kernel in front of it wrote their sums.
template <int C>
cudaError_t launch_join(const Geo &g, const Call &c, int E, bool finals, const Carry &y, int dir,
                        const Carry *y2 = nullptr) {
    Joins j{};
    j.j[0] = Join{y, dir, finals};
    if (y2) j.j[1] = Join{*y2, -dir, finals};
    const dim3 grid(g.W + (g.cu ? g.N : 0), E / (1024 * kJoinVecs), y2 ? 2 : 1);
    return launch_after(la_join_kernel<C>, grid, 256, 0, c.st, g, j, c.log_decay, E, c.slots, c.num_slots);
}

// Where nothing is cut the join has only empty packed sequences' states to hand through, and their
// entries of a slot table to check where the walk does not.
template <int C>
cudaError_t launch_empty(const Geo &g, const Carry &y, const Call &c, int E, bool check) {
    if (!g.cu || !y.last || (y.last == y.s0 && !check)) return cudaSuccess;
    Geo none = g;
    none.W = 0;
    Joins j{};
    j.j[0] = Join{y, 1, 0};
    la_join_kernel<C><<<dim3(g.N, E / (1024 * kJoinVecs)), 256, 0, c.st>>>(none, j, c.log_decay, E, c.slots, c.num_slots);
    return cudaGetLastError();
}

// after: behind another kernel of the call
template <int DAB, int DC, typename Tin, int DIR, bool WALK>
cudaError_t launch_simt(const Geo &g, const Walk &wk, const Call &c, bool after = true) {
    constexpr size_t smem = SimtSmem<DAB, DC>::bytes;
    auto kern = la_simt_kernel<DAB, DC, Tin, DIR, WALK>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (after) return launch_after(kern, g.W, 256, smem, c.st, g, wk, c.log_decay, c.slots, c.num_slots);
    kern<<<g.W, 256, smem, c.st>>>(g, wk, c.log_decay, c.slots, c.num_slots);
    return cudaGetLastError();
}

// Forward: first pass, join, walk.
template <int DK, int DV, typename Tin>
cudaError_t simt_forward(const Call &c, const void *q, const void *k, const void *v, const float *s0, void *o,
                         float *last, float *ws) {
    const Geo g = geo_of<kSimtC>(c, 1, 1, false);
    Walk wk{q, k, v, o, carry_at(ws, g.W, DK * DV), false};
    wk.y.s0 = s0;
    wk.y.last = last;
    // a pool is read and written by different CTAs of the walk: it reads cut sequences' states from a copy
    if (c.slots) wk.y.s0_copy = ws + (size_t)3 * g.W * DK * DV;
    cudaError_t e;
    const bool cut = cuts<kSimtC>(g);
    if (cut) {
        if ((e = launch_simt<DK, DV, Tin, 1, false>(g, wk, c, false)) != cudaSuccess) return e;
        if ((e = launch_join<kSimtC>(g, c, DK * DV, false, wk.y, 1)) != cudaSuccess) return e;
    } else if ((e = launch_empty<kSimtC>(g, wk.y, c, DK * DV, c.slots != nullptr)) != cudaSuccess) {
        return e;
    }
    return launch_simt<DK, DV, Tin, 1, true>(g, wk, c, cut);
}

// Backward: dq walks forwards on S^T; dk and dv backwards on X, whose last state is dinit.
template <int DK, int DV, typename Tin>
cudaError_t simt_backward(const Call &c, const void *q, const void *k, const void *v, const void *d_o, const float *s0,
                          const float *dlast, void *dq, void *dk, void *dv, float *dinit, float *ws) {
    const Geo g = geo_of<kSimtC>(c, 3, 2, false);
    constexpr int E = DK * DV;
    Carry fwd = carry_at(ws, g.W, E), bwd = carry_at(ws + (size_t)3 * g.W * E, g.W, E);
    fwd.s0 = s0;
    bwd.s0 = dlast;
    bwd.last = dinit;
    const Walk sum_f{nullptr, k, v, nullptr, fwd, false}, sum_b{nullptr, q, d_o, nullptr, bwd, false};
    cudaError_t e;
    const bool cut = cuts<kSimtC>(g);
    if (cut) {
        if ((e = launch_simt<DK, DV, Tin, 1, false>(g, sum_f, c, false)) != cudaSuccess) return e;
        if ((e = launch_simt<DK, DV, Tin, -1, false>(g, sum_b, c)) != cudaSuccess) return e;
        if ((e = launch_join<kSimtC>(g, c, E, false, fwd, 1, &bwd)) != cudaSuccess) return e;
    } else if ((e = launch_empty<kSimtC>(g, bwd, c, E, false)) != cudaSuccess) {
        return e;
    }
    Carry bwd_t = bwd;
    bwd_t.last = nullptr;
    if ((e = launch_simt<DV, DK, Tin, 1, true>(g, Walk{d_o, v, k, dq, fwd, true}, c, cut)) != cudaSuccess) return e;
    if ((e = launch_simt<DV, DK, Tin, -1, true>(g, Walk{v, d_o, q, dk, bwd_t, true}, c)) != cudaSuccess) return e;
    return launch_simt<DK, DV, Tin, -1, true>(g, Walk{k, q, d_o, dv, bwd, false}, c);
}

}  // namespace la
}  // namespace kda

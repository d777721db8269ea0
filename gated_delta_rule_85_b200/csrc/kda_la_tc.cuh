// Linear attention with a decay for each head on sm_100a tensor cores (tcgen05, fp32
// accumulation in TMEM), bf16 inputs: the first pass (la_sum_kernel) and the walk
// (la_walk_kernel) of kda_la.cuh, 128 tokens a chunk.
//
// The decay is one constant rate per head, so nothing has to be scaled before a score
// product: a pair's power g^|i-j| is applied to the fp32 score, a row's power to the
// fp32 accumulators, and only the rows that are summed into the state are scaled as
// operands.  Powers never exceed 1; one that underflows stands for a term that small.
//
// Roundings.  Scores (after their power) and the state that a chunk's rows read are
// rounded to bf16, each once; the output is rounded once more.  The state itself is fp32:
// products of bf16 numbers are exact in fp32, but a weighted row g^e b_j is not a bf16
// number, so it is split into bf16 terms that are multiplied in turn into one fp32
// accumulator: three terms (24 bits) where the sum becomes a state that the caller gets or
// another span starts from, two (16 bits, far inside the rounding of the state that rows
// read) elsewhere.  So the walk takes three terms only for sequences that lie in one span;
// the states of cut ones are made by the first pass and the join.
#pragma once

#include <type_traits>

#include "kda_la.cuh"
#include "kda_launch.cuh"
#include "tc_ptx.cuh"
#include "tc_tile.cuh"

namespace kda {
namespace la {

// Measured, 8192 tokens x 32 heads of 128 x 128 (148 spans of 13.8 chunks): first pass 45 us (130 MB
// of k and v; shared memory binds it, see below), walk 70 us (200 MB in, 67 MB out; per chunk
// 2.6 k cycles of products and 4.6 k of shared-memory traffic inside a serial part of 5.5 k of 7 k).
constexpr int kC = 128;                  // tokens of a chunk
constexpr int kBox = 64;                 // token rows of a TMA box
constexpr int kSumWarps = 8;                        // split warps of the first pass, and as many that add up
constexpr int kSumThreads = 64 + 2 * kSumWarps * 32;   // producer, MMA, split, sum
constexpr int kStateWarps = 8;
constexpr int kWalkThreads = 192 + kStateWarps * 32;   // producer, MMA, four output warps, state warps
constexpr int kOutBox = 32;              // token rows of an output box: one warp's

// Waits are bounded, and a warp gives up as a whole.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, ptx::mbar_wait_tries(bar, parity));
}
// One warp of a group polls, the others sleep on a hardware barrier: polling warps take issue
// slots from working ones (measured: more instructions than the work itself).  The barrier also
// hands round whether the poll succeeded, so that no warp is left waiting.
template <int ID, int THREADS>
__device__ __forceinline__ bool wait_group(bool leader, uint32_t bar, uint32_t parity) {
    uint32_t ok = 1;
    if (leader) ok = wait_warp(bar, parity);
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %0, 0;\n\t"
        "barrier.cta.red.and.pred p, %1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "+r"(ok)
        : "n"(ID), "n"(THREADS)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// 16-byte group g of row r in a 128-byte-swizzled atom (64 bf16 wide)
__device__ __forceinline__ uint32_t swz(int r, int g) { return (uint32_t)(r * 128 + ((g ^ (r & 7)) << 4)); }

// A token's weight, and its leading two bf16 terms, each twice.
struct Weight {
    float w;
    __nv_bfloat162 w0, w1;
    __device__ __forceinline__ explicit Weight(float x) : w(x) {
        const float a = __bfloat162float(__float2bfloat16_rn(x));
        w0 = __float2bfloat162_rn(a);
        w1 = __float2bfloat162_rn(x - a);
    }
};
__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// upper halves of two fp32 as two bf16, and what is left without them
__device__ __forceinline__ uint32_t tops(float2 a) {
    return __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x7632);
}
__device__ __forceinline__ float2 rest(float2 a) {
    return ptx::add2(a, make_float2(-hi_bf16(__float_as_uint(a.x)), -hi_bf16(__float_as_uint(a.y))));
}

// Eight weighted elements as bf16 terms, largest first.
// Three: the 24 bits of the fp32 product, cut in three without an error.  (In bf16 arithmetic,
// with residuals by fused multiply-adds and a two-sum, 12 instructions a pair, a 64-token tile
// took 1.6k cycles: bf16 arithmetic runs at a fraction of the rate of moves and fp32.)
// Two: w0 x = t0 + r exactly, by a fused multiply-add, and t1 = round(w1 x + r); what is
// dropped is below 2^-16 of w x.
template <bool THREE>
__device__ __forceinline__ void split8(const uint4 &x, const Weight &w, uint4 &t0, uint4 &t1, uint4 &t2) {
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (THREE) {
            const float2 a = ptx::mul2(make_float2(lo_bf16(in[i]), hi_bf16(in[i])), make_float2(w.w, w.w));
            const float2 b = rest(a), c = rest(b);
            o[0][i] = tops(a);
            o[1][i] = tops(b);
            o[2][i] = tops(c);
        } else {
            const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&in[i]);
            const __nv_bfloat162 a = __hmul2_rn(w.w0, v), b = __hfma2(w.w1, v, __hfma2(w.w0, v, __hneg2(a)));
            o[0][i] = *reinterpret_cast<const uint32_t *>(&a);
            o[1][i] = *reinterpret_cast<const uint32_t *>(&b);
            o[2][i] = 0u;
        }
    }
    t0 = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
    t1 = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
    t2 = make_uint4(o[2][0], o[2][1], o[2][2], o[2][3]);
}

// ------------------------------------------------------------------ first pass

// Sums of b c^T over the parts of cut sequences that lie in a span: of the one that goes on
// behind the span in walking order (sum_out, or sum_in when it came from the span before
// too), and with final states wanted of the one that came from before and ends in it
// (sum_in).  The tokens of a part are contiguous: the CTA runs over them in tiles of 64 from
// the far end towards the near one, against the walk, and takes the far part first, so that
// what the walk reads first is what L2 saw last.
//
// Weighted rows are three terms where these sums can become a state that the caller gets (asked
// for or not: the outputs do not depend on that), else two.  A tile's products
// leave TMEM after 8 or 12 K steps and are added in fp32 registers, scaled by the decay of the tokens behind the tile, so that neither the tensor core's
// accumulation nor a product of many decays costs fp32 accuracy over long sequences.
struct SumRole {
    CUtensorMap b, c;
    float *sum_in, *sum_out;
    int dir;
    int three;          // terms of a weighted row: three, or two
    int want_last;
};
struct SumArgs {
    SumRole role[2];
};

template <int DB, int DC>
struct SumSmem {
    static constexpr int BT = DB * kBox * 2, CT = DC * kBox * 2;   // bytes of a 64-token tile
    static constexpr int STAGE = BT + CT;
    static constexpr int NST = 4;
    static constexpr int E = NST * STAGE;                // [2][middle, low] terms of c
    static constexpr int BAR = E + 2 * 2 * CT;
    static constexpr int BYTES = BAR + 8 * (2 * NST + 4 + 1) + 16;
    static constexpr int ALLOC = BYTES + 1024;
    static_assert(ALLOC <= 232448, "shared memory");
};

template <int DB, int DC>
__global__ void __launch_bounds__(kSumThreads, 1)
la_sum_kernel(const __grid_constant__ SumArgs args, Geo g, const float *__restrict__ log_decay) {
    using L = SumSmem<DB, DC>;
    constexpr int NST = L::NST;
    let_next_start();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = ptx::smem_u32(sm);
    const uint32_t bar_full = sb + L::BAR, bar_done = bar_full + 8 * NST, bar_ready = bar_done + 8 * NST,
                   bar_added = bar_ready + 16, bar_fin = bar_added + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::BAR + 8 * (2 * NST + 5));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SumRole &role = args.role[blockIdx.y];
    const int dir = role.dir, w = blockIdx.x;
    const long long lo = g.lo(w), hi = g.hi(w);
    // the far part, then the near one: tokens [ta, tb) in nt tiles, counted from the far end
    struct Part {
        long long ta, tb;
        int h, nt;
        bool in;   // came from the span before
    } part[2];
    part[0] = part[1] = Part{0, 0, 0, 0, false};
    {
        Cursor<kC> cur;
        const long long edge = dir > 0 ? hi - 1 : lo;
        cur.seek(g, edge);
        bool through = false;
        if (cur.valid && cur.c != (dir > 0 ? cur.nck - 1 : 0)) {
            const long long u_near = dir > 0 ? edge - cur.c : edge + (cur.nck - 1 - cur.c);
            through = dir > 0 ? u_near < lo : u_near >= hi;
            const long long near = through ? (dir > 0 ? lo : hi - 1) : u_near;
            Part &p = part[0];
            p.ta = dir > 0 ? cur.tok() - (edge - near) * kC : cur.tok();
            p.tb = dir > 0 ? cur.tok() + kC : min(cur.t1, cur.tok() + (near - edge + 1) * kC);
            p.h = cur.h;
            p.in = through;
        }
        if (role.want_last && !through) {
            cur.seek(g, dir > 0 ? lo : hi - 1);
            // it came from before, and its end (all of it that is left) lies in the span
            const int left = dir > 0 ? cur.nck - 1 - cur.c : cur.c;
            if (cur.valid && cur.c != (dir > 0 ? 0 : cur.nck - 1) && left < hi - lo) {
                Part &p = part[1];
                p.ta = dir > 0 ? cur.tok() : cur.t0;
                p.tb = dir > 0 ? cur.t1 : min(cur.t1, cur.tok() + kC);
                p.h = cur.h;
                p.in = true;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) part[x].nt = (int)((part[x].tb - part[x].ta + kBox - 1) / kBox);
    }
    const int nt = part[0].nt + part[1].nt;
    if (nt == 0) return;   // nothing cut
    // first token of tile x; only a part's last tile in time can be shorter than 64
    auto tile_tok = [&](const Part &p, int x) { return p.ta + (long long)(dir > 0 ? p.nt - 1 - x : x) * kBox; };

    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tslot), 256);
        ptx::tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_done + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(bar_ready + 8 * s, kSumWarps);
            ptx::mbar_init(bar_added + 8 * s, kSumWarps);
        }
        ptx::mbar_init(bar_fin, 1);
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tslot;
    bool ok = true;

    if (warp == 0) {
        // ---------------- producer
        int n = 0;
        for (; n < nt; ++n) {
            const int s = n % NST;
            if (n >= NST && !(ok = wait_warp(bar_done + 8 * s, (uint32_t)((n / NST - 1) & 1)))) break;
            if (lane == 0) {
                const uint32_t bar = bar_full + 8 * s, dst = sb + s * L::STAGE;
                const bool far = n < part[0].nt;
                const Part &p = far ? part[0] : part[1];
                const int t = (int)tile_tok(p, far ? n : n - part[0].nt);
                ptx::mbar_arrive_expect_tx(bar, L::STAGE);
#pragma unroll
                for (int a = 0; a < DB / 64; ++a) ptx::tma_load_3d(dst + a * 8192, &role.b, bar, a * 64, p.h, t);
#pragma unroll
                for (int a = 0; a < DC / 64; ++a)
                    ptx::tma_load_3d(dst + L::BT + a * 8192, &role.c, bar, a * 64, p.h, t);
            }
            __syncwarp();
        }
        if (!ok) {
            if (lane == 0) flag_status(KDA_DEV_WAIT_TIMEOUT);
            for (int k = max(0, n - NST); k < n; ++k)   // copies in flight
                wait_warp(bar_full + 8 * (k % NST), (uint32_t)((k / NST) & 1));
        }
    } else if (warp == 1) {
        // ---------------- MMA
        constexpr uint32_t id = ptx::idesc_bf16_f32(128, DC, true, true);
        for (int n = 0; n < nt; ++n) {
            const int s = n % NST, e = n & 1;
            ok = wait_warp(bar_full + 8 * s, (uint32_t)((n / NST) & 1)) &&
                 wait_warp(bar_ready + 8 * e, (uint32_t)((n >> 1) & 1)) &&
                 (n < 2 || wait_warp(bar_added + 8 * e, (uint32_t)(((n >> 1) - 1) & 1)));
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t bt = sb + s * L::STAGE;
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    if (p == 2 && !role.three) break;
                    const uint32_t ct = p == 0 ? bt + L::BT : sb + L::E + (e * 2 + p - 1) * L::CT;
#pragma unroll
                    for (int ks = 0; ks < kBox / 16; ++ks)
                        ptx::mma_bf16(tmem + e * 128, ptx::desc_mnmajor_sw128(bt + ks * 2048, 8192, 1024),
                                      ptx::desc_mnmajor_sw128(ct + ks * 2048, 8192, 1024), id, p + ks > 0);
                }
                ptx::mma_commit(bar_done + 8 * s);
            }
            __syncwarp();
        }
        if (lane == 0) {   // products in flight
            if (!ok) flag_status(KDA_DEV_WAIT_TIMEOUT);
            ptx::mma_commit(bar_fin);
        }
        __syncwarp();
        wait_warp(bar_fin, 0u);
    } else if (warp < 2 + kSumWarps) {
        // ---------------- split the weighted rows.  Thread <-> token row, a part of its columns.
        constexpr int JP = kSumWarps / 2, CG = DC / 8 / JP, BG = DB / 8 / JP;   // 16-byte groups
        const int ct = tid - 64, jr = ct & 63, jq = ct >> 6;
        auto wait_split = [&](uint32_t bar, uint32_t parity) {
            return wait_group<1, kSumWarps * 32>(warp == 2, bar, parity);
        };
        int n = 0;
#pragma unroll 1
        for (int q = 0; q < 2 && ok; ++q) {
            const Part &p = part[q];
            if (p.nt == 0) continue;
            const double lg = (double)rate_of(log_decay, p.h);
            // forwards the weight counts from the tile's end, backwards from its start
            const Weight full_wt((float)exp64(lg * (dir > 0 ? kBox - 1 - jr : jr + 1)));
#pragma unroll 1
            for (int x = 0; x < p.nt; ++x, ++n) {
                const int s = n % NST, e = n & 1;
                // the tile is there, and the smaller terms' buffer was multiplied
                ok = wait_split(bar_full + 8 * s, (uint32_t)((n / NST) & 1)) &&
                     (n < 2 || wait_split(bar_done + 8 * ((n - 2) % NST), (uint32_t)(((n - 2) / NST) & 1)));
                if (!ok) break;
                const int len = (int)min((long long)kBox, p.tb - tile_tok(p, x));
                const uint32_t bt = sb + s * L::STAGE, c0 = bt + L::BT;
                const uint32_t c1 = sb + L::E + e * 2 * L::CT, c2 = c1 + L::CT;
                const bool live = jr < len;
                Weight wt = full_wt;
                if (len < kBox && dir > 0) wt = Weight(live ? (float)exp64(lg * (len - 1 - jr)) : 0.f);
                uint4 v[CG];   // the row's groups
                uint32_t at[CG];
#pragma unroll
                for (int k = 0; k < CG; ++k) {
                    const int cg = jq * CG + k;
                    at[k] = (cg >> 3) * 8192 + swz(jr, cg & 7);
                    v[k] = ptx::lds128(c0 + at[k]);
                    if (!live) v[k] = make_uint4(0, 0, 0, 0);   // rows behind the end may hold anything
                }
                auto put = [&](auto three) {
#pragma unroll
                    for (int k = 0; k < CG; ++k) {
                        uint4 t0, t1, t2;
                        split8<decltype(three)::value>(v[k], wt, t0, t1, t2);
                        ptx::sts128(c0 + at[k], t0);
                        ptx::sts128(c1 + at[k], t1);
                        if (decltype(three)::value) ptx::sts128(c2 + at[k], t2);
                    }
                };
                if (role.three) put(std::true_type());
                else put(std::false_type());
                if (!live)
#pragma unroll
                    for (int k = 0; k < BG; ++k) {
                        const int cg = jq * BG + k;
                        ptx::sts128(bt + (cg >> 3) * 8192 + swz(jr, cg & 7), 0, 0, 0, 0);
                    }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_ready + 8 * e);
            }
        }
        if (!ok && lane == 0) flag_status(KDA_DEV_WAIT_TIMEOUT);
    } else {
        // ---------------- add up the tiles' sums.  Thread <-> state row, half of its columns.
        constexpr int CPT = DC / (kSumWarps / 4);
        const int quad = warp & 3, row = quad * 32 + lane, col = ((warp - 2 - kSumWarps) >> 2) * CPT;
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16) + col;
        float S[CPT];
        int n = 0;
#pragma unroll 1
        for (int q = 0; q < 2 && ok; ++q) {
            const Part &p = part[q];
            if (p.nt == 0) continue;
#pragma unroll
            for (int x = 0; x < CPT; ++x) S[x] = 0.f;
            const double lg = (double)rate_of(log_decay, p.h), full_dec = exp64(lg * kBox);
            double behind = 1.0;         // decay of the tokens behind the tile
#pragma unroll 1
            for (int x = 0; x < p.nt; ++x, ++n) {
                const int len = (int)min((long long)kBox, p.tb - tile_tok(p, x));
                const float sc = (float)behind;
                behind *= len == kBox ? full_dec : exp64(lg * len);
                ok = wait_group<2, kSumWarps * 32>(warp == 2 + kSumWarps, bar_done + 8 * (n % NST),
                                                   (uint32_t)((n / NST) & 1));
                if (!ok) break;
                ptx::tc_fence_after();
                if (quad * 32 < DB) {
                    const uint32_t u = tl + (n & 1) * 128;
#pragma unroll
                    for (int k = 0; k < CPT / 16; ++k) {
                        float v[16];
                        ptx::tmem_ld16(u + 16 * k, v);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) S[16 * k + i] = fmaf(sc, v[i], S[16 * k + i]);
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_added + 8 * (n & 1));
            }
            if (ok && row < DB) {
                float *dst = (p.in ? role.sum_in : role.sum_out) + ((long long)w * DB + row) * DC + col;
#pragma unroll
                for (int x = 0; x < CPT; x += 4) store4(dst + x, make_float4(S[x], S[x + 1], S[x + 2], S[x + 3]));
            }
        }
        if (!ok && lane == 0) flag_status(KDA_DEV_WAIT_TIMEOUT);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 256);
    }
}

// ------------------------------------------------------------------ the walk

// The valid items of one span in walking order, with what every role has to agree on.
struct SpanWalk {
    Cursor<kC> cur;
    long long lo, hi, i;
    int dir;
    bool ends;              // the item is the last of its sequence in walking order
    bool first;             // the first item of a part
    bool from_before;       // its part's sequence started in an earlier span
    bool whole;             // its sequence lies in this span from start to end
    bool fresh;

    __device__ __forceinline__ SpanWalk(const Geo &g, int w, int dir_) : lo(g.lo(w)), hi(g.hi(w)), i(-1), dir(dir_) {
        cur = Cursor<kC>{};
        ends = first = from_before = whole = false;
        fresh = true;
    }
    __device__ __forceinline__ bool next(const Geo &g) {
        while (++i < hi - lo) {
            const int c = cur.c + dir;
            if (cur.valid && c >= 0 && c < cur.nck) {
                cur.c = c;
            } else {
                cur.seek(g, dir > 0 ? lo + i : hi - 1 - i);
                if (!cur.valid) continue;
            }
            const bool begins = cur.c == (dir > 0 ? 0 : cur.nck - 1);
            ends = cur.c == (dir > 0 ? cur.nck - 1 : 0);
            from_before = fresh && !begins;
            first = fresh || begins;
            if (first) whole = begins && (dir > 0 ? cur.nck - 1 - cur.c : cur.c) < hi - lo - i;
            fresh = false;
            return true;
        }
        return false;
    }
    // the chunk's U is needed: by the part's next chunk, or for a final state that the walk writes
    __device__ __forceinline__ bool need_u(bool want_last) const {
        return !(ends || i == hi - lo - 1) || (ends && whole && want_last);
    }
};

// A chunk as the producer hands it to the other warps, in the ring entry of its stage: seen by
// whoever has waited for the stage's tiles, and read before its products free the stage.  (Each role
// walking the span by itself took 20 registers a thread, and spilled.)
struct __align__(16) Item {
    long long tok;      // first token
    int h, n;           // head, sequence
    int len;            // tokens; 0: the span has ended
    int flags;
    int pad[2];
    static constexpr int FIRST = 1, FROM_BEFORE = 2, WHOLE = 4, ENDS = 8, NEED_U = 16;   // as in SpanWalk
    __device__ __forceinline__ bool is(int f) const { return flags & f; }
};

struct WalkRole {
    CUtensorMap a, b, c, out_map;
    __nv_bfloat16 *out;
    Carry y;
    int dir;
    int three;          // states of whole sequences are the caller's: three terms (asked for or not)
    int transposed;     // the carried states are [DC][DAB]; y.last is null then
};
struct WalkArgs {
    WalkRole role[3];
};

template <int DAB, int DC>
struct WalkSmem {
    static constexpr int AT = DAB * kC * 2, CT = DC * kC * 2;   // bytes of a chunk's tile
    static constexpr int STAGE = 2 * AT + CT;
    static constexpr int ROOM = 229376 - AT;
    static constexpr int NST = ROOM / STAGE < 4 ? ROOM / STAGE : 4;
    // The bf16 state, then the low terms of b.  It lies before the stages: an M = 128 operand of
    // 64 state rows reads 16 KB on from its tile (the product's lanes 64.. are not used), which
    // must stay inside the allocation -- from here into stage 0, from a stage's tile into its next.
    static constexpr int X = 0;
    static constexpr int ST0 = AT;
    static constexpr int BAR = ST0 + NST * STAGE;
    static constexpr int ITEM = BAR + ((8 * (3 * NST + 9) + 16 + 15) & ~15);
    static constexpr int BYTES = ITEM + NST * (int)sizeof(Item);
    static constexpr int ALLOC = BYTES + 1024;
    static_assert(NST >= 2 && ALLOC <= 232448, "shared memory");
};

// One span of one walk.  Per chunk, with the state S that it starts from:
//   scores = A B^T            -> P: the powers and the mask on the fp32 scores, bf16, in TMEM
//   inter  = A bf16(S)
//   U      = (weights B)^T C  -> S <- g^len S + U in fp32 registers
//   intra  = P C              -> out = intra + powers inter
// Warps: 0 loads (TMA, NST chunks ahead), 1 issues every MMA, 2-5 turn scores into P and
// accumulators into rows of the output, 6-13 weigh the b rows and carry the state (thread
// <-> state row and half of its columns).  Once inter is done the tiles of A and of the
// bf16 state are free until the chunk's U is: they take the middle and low terms of b.
// TMEM columns: scores, then P over them [0, 128), intra [128, 256), inter [256, 384), U [384, 512).
template <int DAB, int DC>
__global__ void __launch_bounds__(kWalkThreads, 1)
la_walk_kernel(const __grid_constant__ WalkArgs args, Geo g, const float *__restrict__ log_decay,
               const int32_t *__restrict__ slots, int num_slots, int roles) {
    using L = WalkSmem<DAB, DC>;
    constexpr int NST = L::NST;
    let_next_start();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = ptx::smem_u32(sm);
    const uint32_t bar_full = sb + L::BAR, bar_free = bar_full + 8 * NST, bar_out = bar_free + 8 * NST,
                   bar_sc = bar_out + 8 * NST, bar_in = bar_sc + 8, bar_p = bar_in + 8, bar_b = bar_p + 8, bar_u = bar_b + 8, bar_o = bar_u + 8,
                   bar_x = bar_o + 8, bar_od = bar_x + 8, bar_fin = bar_od + 8;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::BAR + 8 * (3 * NST + 9));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the roles of one span run side by side: they share most of their tiles in L2
    const WalkRole &role = args.role[blockIdx.x % roles];
    const int dir = role.dir, w = blockIdx.x / roles;
    const Carry &y = role.y;
    const bool want_last = y.last != nullptr;

    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_free + 8 * s, 1);
            ptx::mbar_init(bar_out + 8 * s, 4);
        }
        ptx::mbar_init(bar_sc, 1);
        ptx::mbar_init(bar_in, 1);
        ptx::mbar_init(bar_p, 4);
        ptx::mbar_init(bar_b, kStateWarps);
        ptx::mbar_init(bar_u, 1);
        ptx::mbar_init(bar_o, 1);
        ptx::mbar_init(bar_x, kStateWarps);
        ptx::mbar_init(bar_od, 4);
        ptx::mbar_init(bar_fin, 1);
        ptx::fence_mbar_init();
    }
    // before any tensor memory is taken: what waits holds nothing that the kernels it waits for may need
    wait_for_previous();
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tslot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tslot;
    const uint32_t t_sc = tmem, t_oa = tmem + 128, t_oi = tmem + 256, t_u = tmem + 384;
    bool ok = true;
    int n = 0;   // chunks so far
    Item *items = reinterpret_cast<Item *>(sm + L::ITEM);
    // chunk k's entry, once `full` of its stage was waited for
    auto item_of = [&](int k) {
        const uint32_t at = sb + L::ITEM + (uint32_t)(k % NST) * (uint32_t)sizeof(Item);
        const uint4 a = ptx::lds128(at), b = ptx::lds128(at + 16);
        Item x;
        x.tok = (long long)(((unsigned long long)a.y << 32) | a.x);
        x.h = (int)a.z;
        x.n = (int)a.w;
        x.len = (int)b.x;
        x.flags = (int)b.y;
        return x;
    };

    if (warp == 0) {
        // ---------------- producer, and the sender of outputs
        int meta[NST][3] = {};   // lane 0: first token, head and length of the chunks in flight
        // The output rows of chunk k are in its tile: send the whole boxes, and wait until they are read.
        // (A box in which a sequence ends was written by its warp: the rows behind it are not its.)
        auto send = [&](int k) {
            const int s = k % NST;
            if (!wait_warp(bar_out + 8 * s, (uint32_t)((k / NST) & 1))) return false;
            if (lane == 0) {
#pragma unroll
                for (int x = 0; x < NST; ++x)
                    if (x == s)
                        for (int q = 0; q * kOutBox + kOutBox <= meta[x][2]; ++q)
#pragma unroll
                            for (int a = 0; a < DC / 64; ++a)
                                ptx::tma_store_3d(&role.out_map, sb + L::ST0 + s * L::STAGE + a * 16384 + q * kOutBox * 128,
                                                  a * 64, meta[x][1], meta[x][0] + q * kOutBox);
                ptx::bulk_commit();
                ptx::bulk_wait_read_all();
            }
            __syncwarp();
            return true;
        };
        SpanWalk it(g, w, dir);
        while (true) {
            const bool have = it.next(g);
            const int s = n % NST;
            const uint32_t bar = bar_full + 8 * s, dst = sb + L::ST0 + s * L::STAGE, old = (uint32_t)((n / NST - 1) & 1);
            const int len = have ? it.cur.len() : 0, t = (int)it.cur.tok(), h = it.cur.h;
            const int boxes = len > kBox ? 2 : 1;
            auto load = [&](const CUtensorMap *map, uint32_t at, int atoms) {
                for (int x = 0; x < boxes; ++x)
                    for (int a = 0; a < atoms; ++a)
                        ptx::tma_load_3d(at + a * 16384 + x * 8192, map, bar, a * 64, h, t + x * kBox);
            };
            // the last product frees C (and B); the tiles that the output goes through are free once it is out
            constexpr bool B_EARLY = DC <= DAB;
            if (n >= NST && !(ok = wait_warp(bar_free + 8 * s, old))) break;
            if (lane == 0) {
                Item x;
                x.tok = it.cur.tok();
                x.h = h;
                x.n = it.cur.n;
                x.len = len;
                x.flags = (it.first ? Item::FIRST : 0) | (it.from_before ? Item::FROM_BEFORE : 0) |
                          (it.whole ? Item::WHOLE : 0) | (it.ends ? Item::ENDS : 0) |
                          (it.need_u(want_last) ? Item::NEED_U : 0);
                x.pad[0] = x.pad[1] = 0;
                items[s] = x;
                if (have) {
                    ptx::mbar_arrive_expect_tx(bar, (uint32_t)(L::STAGE / 2 * boxes));
                    if (B_EARLY) load(&role.b, dst + L::AT, DAB / 64);
                    load(&role.c, dst + 2 * L::AT, DC / 64);
                } else {
                    ptx::mbar_arrive(bar);
                }
            }
            __syncwarp();
            if (!have) break;
            if (n >= NST) ok = send(n - NST);
            // (after a wait that ran out the rest is loaded all the same: the barrier has counted it)
            if (lane == 0) {
                load(&role.a, dst, DAB / 64);
                if (!B_EARLY) load(&role.b, dst + L::AT, DAB / 64);
                meta[n % NST][0] = t;
                meta[n % NST][1] = h;
                meta[n % NST][2] = len;
            }
            __syncwarp();
            ++n;
            if (!ok) break;
        }
        for (int k = max(0, n - NST); k < n && ok; ++k) ok = send(k);
        if (!ok) {
            if (lane == 0) flag_status(KDA_DEV_WAIT_TIMEOUT);
            for (int k = max(0, n - NST); k < n; ++k)   // copies in flight
                wait_warp(bar_full + 8 * (k % NST), (uint32_t)((k / NST) & 1));
        }
    } else if (warp == 1) {
        // ---------------- MMA
        constexpr uint32_t id_sc = ptx::idesc_bf16_f32(128, 128), id_in = ptx::idesc_bf16_f32(128, DC, false, true),
                           id_u = ptx::idesc_bf16_f32(128, DC, true, true);
        const uint32_t me = lane == 0 ? 1u : 0u;
        // (values that a shuffle hands round are uniform to the compiler)
        const uint32_t sbu = __shfl_sync(0xffffffffu, sb, 0), tmu = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t u_sc = tmu, u_oa = tmu + 128, u_oi = tmu + 256, u_u = tmu + 384;
        while (true) {
            const int s = __shfl_sync(0xffffffffu, n % NST, 0);
            const uint32_t at = sbu + L::ST0 + s * L::STAGE, bt = at + L::AT, ct = bt + L::AT, ph = (uint32_t)(n & 1);
            // scores: the region is free once the chunk before has multiplied its P
            if (!(ok = wait_warp(bar_full + 8 * s, (uint32_t)((n / NST) & 1)))) break;
            const Item item = item_of(n);
            if (item.len == 0) break;
            if (n > 0 && !(ok = wait_warp(bar_o, ph ^ 1u))) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < DAB / 16; ++ks)
                ptx::mma_bf16_elected(me, u_sc, kda::tc::kdesc(at, ks, kC), kda::tc::kdesc(bt, ks, kC), id_sc, ks > 0);
            ptx::mma_commit_elected(me, bar_sc);
            ok = wait_warp(bar_x, ph) && (n == 0 || wait_warp(bar_od, ph ^ 1u));
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < DAB / 16; ++ks)
                ptx::mma_bf16_elected(me, u_oi, kda::tc::kdesc(at, ks, kC),
                                      ptx::desc_mnmajor_sw128(sbu + L::X + ks * 2048, DAB * 128, 1024), id_in, ks > 0);
            ptx::mma_commit_elected(me, bar_in);
            if (!(ok = wait_warp(bar_b, ph))) break;
            ptx::tc_fence_after();
            if (item.is(Item::NEED_U)) {
                const bool three = role.three && item.is(Item::WHOLE);
                // small terms first: the accumulator is least rounded while it is small
#pragma unroll 1
                for (int x = three ? 0 : 1; x < 3; ++x) {
                    const uint32_t term = __shfl_sync(0xffffffffu, x == 0 ? sbu + L::X : x == 1 ? at : bt, 0);
                    const uint32_t acc = x > (three ? 0 : 1) ? 1u : 0u;
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks)
                        ptx::mma_bf16_elected(me, u_u, ptx::desc_mnmajor_sw128(term + ks * 2048, 16384, 1024),
                                              ptx::desc_mnmajor_sw128(ct + ks * 2048, 16384, 1024), id_u,
                                              ks > 0 ? 1u : acc);
                }
                ptx::mma_commit_elected(me, bar_u);
            }
            if (!(ok = wait_warp(bar_p, ph))) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < kC / 16; ++ks)
                ptx::mma_bf16_ts_elected(me, u_oa, u_sc + ks * 8, ptx::desc_mnmajor_sw128(ct + ks * 2048, 16384, 1024),
                                         id_in, ks > 0);
            ptx::mma_commit_elected(me, bar_o);
            ptx::mma_commit_elected(me, bar_free + 8 * s);
            ++n;
        }
        if (lane == 0) {   // products in flight
            if (!ok) flag_status(KDA_DEV_WAIT_TIMEOUT);
            ptx::mma_commit(bar_fin);
        }
        __syncwarp();
        wait_warp(bar_fin, 0u);
    } else if (warp < 6) {
        // ---------------- scores -> P, accumulators -> out.  Thread <-> row i.
        const int quad = warp & 3, i = quad * 32 + lane;
        if (g.cu && slots) check_slots(g.N, slots, num_slots, tid - 64, 128);
        auto wait_out = [&](uint32_t bar, uint32_t parity) { return wait_group<1, 128>(warp == 2, bar, parity); };
        const uint32_t tl = (uint32_t)(quad * 32) << 16;
        // Powers that a head keeps: in a 16-column block all on one side of the diagonal
        // g^|i-j| = g^(distance to the block's nearest column) step[m]; in the row's own block it is
        // near[m].  P and out are rounded to bf16, which a fast exponential's error does not reach.
        float step[16], near[16];
        float l2 = 0.f;   // log2 g
        const int li = i & 15, bi = i >> 4;
        int head = -1;
        while (true) {
            const uint32_t ph = (uint32_t)(n & 1);
            if (!(ok = wait_out(bar_full + 8 * (n % NST), (uint32_t)((n / NST) & 1)))) break;
            const Item item = item_of(n);
            const int h = item.h, len = item.len;
            const long long t = item.tok;
            if (len == 0) break;
            if (h != head) {
                head = h;
                l2 = rate_of(log_decay, h) * 1.44269504f;
#pragma unroll
                for (int m = 0; m < 16; ++m) {
                    step[m] = kda::tc::exp2_fast(l2 * (dir > 0 ? 15 - m : m));
                    near[m] = kda::tc::exp2_fast(l2 * max((li - m) * dir, 0));
                }
            }
            if (!(ok = wait_out(bar_sc, ph))) break;
            ptx::tc_fence_after();
            // 32 score columns a step (P overwrites scores that were read).  The loops over columns stay
            // rolled here: the kernel's steady state has to fit the instruction cache.
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                uint32_t p[16];
                if (dir > 0 ? b > quad : b < quad) {
#pragma unroll
                    for (int x = 0; x < 16; ++x) p[x] = 0u;
                } else {
                    float s[32];
                    ptx::tmem_ld32(t_sc + tl + 32 * b, s);
                    float r[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        r[k] = kda::tc::exp2_fast(l2 * max(dir > 0 ? i - 32 * b - 16 * k - 15 : 32 * b + 16 * k - i, 0));
                    ptx::tmem_wait_ld();
                    if (b != quad && (dir > 0 || 32 * b + 32 <= len)) {   // no row of the warp is masked
#pragma unroll
                        for (int m = 0; m < 32; m += 2) {
                            const float2 c = ptx::mul2(make_float2(step[m & 15], step[(m & 15) + 1]), make_float2(r[m >> 4], r[m >> 4]));
                            const float2 z = ptx::mul2(make_float2(s[m], s[m + 1]), c);
                            p[m / 2] = pack2(z.x, z.y);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // scores on the masked side and behind the end may be anything, and count as zeros
                            const int side = (bi - 2 * b - k) * dir;   // 0: the row's own block, below: masked
                            const int first = side == 0 && dir < 0 ? li : 0;
                            const int last = side < 0 ? -1 : min(side == 0 && dir > 0 ? li : 15, len - 1 - 32 * b - 16 * k);
#pragma unroll
                            for (int m = 0; m < 16; m += 2) {
                                float z[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float c = side == 0 ? near[m + e] : step[m + e] * r[k];
                                    z[e] = m + e >= first && m + e <= last ? s[16 * k + m + e] * c : 0.f;
                                }
                                p[8 * k + m / 2] = pack2(z[0], z[1]);
                            }
                        }
                    }
                }
                ptx::tmem_st16(t_sc + tl + 16 * b, p);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_p);
            if (!(ok = wait_out(bar_o, ph))) break;
            ptx::tc_fence_after();
            // the rows leave through the tile of A (and B): every product of the chunk is done
            const float up = kda::tc::exp2_fast(l2 * (dir > 0 ? i + 1 : max(len - 1 - i, 0)));
            const int s = n % NST;
            const uint32_t tile = sb + L::ST0 + s * L::STAGE;
#pragma unroll 1
            for (int b = 0; b < DC / 32; ++b) {
                float u[32], v[32];
                ptx::tmem_ld32(t_oa + tl + 32 * b, u);
                ptx::tmem_ld32(t_oi + tl + 32 * b, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int e = 8 * x + 2 * k;
                        const float2 z = ptx::fma2(make_float2(up, up), make_float2(v[e], v[e + 1]), make_float2(u[e], u[e + 1]));
                        r[k] = pack2(z.x, z.y);
                    }
                    const int cg = 4 * b + x;
                    ptx::sts128(tile + (cg >> 3) * 16384 + swz(i, cg & 7), r[0], r[1], r[2], r[3]);
                }
            }
            ptx::tc_fence_before();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_od);
            if (quad * kOutBox + kOutBox > len) {   // a sequence ends in these rows
                for (int x = lane; x < kOutBox * (DC / 8); x += 32) {
                    const int r = quad * kOutBox + x / (DC / 8), cg = x % (DC / 8);
                    if (r < len)
                        *reinterpret_cast<uint4 *>(role.out + ((t + r) * g.H + h) * DC + cg * 8) =
                            ptx::lds128(tile + (cg >> 3) * 16384 + swz(r, cg & 7));
                }
                __syncwarp();
            }
            if (lane == 0) ptx::mbar_arrive(bar_out + 8 * s);
            ++n;
        }
        if (!ok && lane == 0) flag_status(KDA_DEV_WAIT_TIMEOUT);
    } else {
        // ---------------- state.  Thread <-> state row, and <-> token row when it weighs b; half of the columns.
        constexpr int SP = kStateWarps / 4, CPT = DC / SP, BG = DAB / 8 / SP;   // state columns, 16-byte groups of a b row
        const int quad = warp & 3, part = (warp - 6) >> 2, r = quad * 32 + lane, col = part * CPT;
        const uint32_t tl = ((uint32_t)(quad * 32) << 16) + col;
        auto wait_state = [&](uint32_t bar, uint32_t parity) {
            return wait_group<2, kStateWarps * 32>(warp == 6, bar, parity);
        };
        const bool has = r < DAB;
        float S[CPT];
        int head = -1, wlen = -1, nu = 0;
        Weight wt(0.f);                          // this token row's
        float2 dec = make_float2(0.f, 0.f);      // decay of the chunk
        while (true) {
            const uint32_t ph = (uint32_t)(n & 1);
            const int s = n % NST;
            if (!(ok = wait_state(bar_full + 8 * s, (uint32_t)((n / NST) & 1)))) break;
            const Item item = item_of(n);
            const int h = item.h, len = item.len;
            if (len == 0) break;
            if (h != head || len != wlen) {
                head = h;
                wlen = len;
                const float lg = rate_of(log_decay, h);
                wt = Weight(r < len ? (float)exp64((double)lg * (dir > 0 ? len - 1 - r : r + 1)) : 0.f);
                dec = decay2(lg, len);
            }
            if (item.is(Item::FIRST)) {
                const float *src = nullptr;
                const int row = state_row(slots, num_slots, item.n, 192);   // (the group's first thread)
                if (item.is(Item::FROM_BEFORE)) src = y.start + (long long)w * DAB * DC;
                else if (y.s0_copy && !item.is(Item::WHOLE)) src = y.s0_copy + ((long long)item.n * g.H + h) * (DAB * DC);
                else if (y.s0 && row >= 0) src = y.s0 + ((long long)row * g.H + h) * (DAB * DC);
                if (!src || !has) {
#pragma unroll
                    for (int x = 0; x < CPT; ++x) S[x] = 0.f;
                } else if (role.transposed) {
#pragma unroll
                    for (int x = 0; x < CPT; ++x) S[x] = src[(col + x) * DAB + r];
                } else {
#pragma unroll
                    for (int x = 0; x < CPT; x += 4) {
                        const float4 v = load4(src + r * DC + col + x);
                        S[x] = v.x; S[x + 1] = v.y; S[x + 2] = v.z; S[x + 3] = v.w;
                    }
                }
            }
            // bf16 state for this chunk's inter product (the chunk before is done with the tile: its U was read,
            // or it needed none and its inter was waited for)
            if (has) {
#pragma unroll
                for (int k = 0; k < CPT / 8; ++k) {
                    const int cg = col / 8 + k;
                    ptx::sts128(sb + L::X + (cg >> 3) * (DAB * 128) + swz(r, cg & 7), pack2(S[8 * k], S[8 * k + 1]),
                                pack2(S[8 * k + 2], S[8 * k + 3]), pack2(S[8 * k + 4], S[8 * k + 5]),
                                pack2(S[8 * k + 6], S[8 * k + 7]));
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_x);
            const uint32_t at = sb + L::ST0 + s * L::STAGE, bt = at + L::AT, ct = bt + L::AT;
            if (r >= len) {   // what lies behind the end may be another sequence's, or anything
#pragma unroll
                for (int k = 0; k < CPT / 8; ++k) {
                    const int cg = col / 8 + k;
                    ptx::sts128(ct + (cg >> 3) * 16384 + swz(r, cg & 7), 0, 0, 0, 0);
                }
            }
            const bool need = item.is(Item::NEED_U), three = role.three && item.is(Item::WHOLE);
            auto group_at = [&](int k) {
                const int cg = part * BG + k;
                return (uint32_t)((cg >> 3) * 16384 + swz(r, cg & 7));
            };
            // two terms: the leading one takes b's place once the scores are done; of the first groups,
            // while inter runs, the second waits in registers for the tile of A (four groups instead of two
            // spill, and the walk of 8192 x 32 heads takes 77 us instead of 74.5)
            constexpr int EG = 2;
            uint4 mid[EG];
            if (need && !three) {
                if (!(ok = wait_state(bar_sc, ph))) break;
#pragma unroll
                for (int k = 0; k < EG; ++k) {
                    uint4 t0, t2, x = ptx::lds128(bt + group_at(k));
                    if (r >= len) x = make_uint4(0, 0, 0, 0);
                    split8<false>(x, wt, t0, mid[k], t2);
                    ptx::sts128(bt + group_at(k), t0);
                }
            }
            // inter done: the tiles of A and X are free
            if (!(ok = wait_state(bar_in, ph))) break;
            if (need && !three) {
#pragma unroll
                for (int k = 0; k < EG; ++k) ptx::sts128(at + group_at(k), mid[k]);
#pragma unroll 1
                for (int k = EG; k < BG; k += 2) {   // (rolled: instruction cache)
                    uint4 x[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) x[z] = ptx::lds128(bt + group_at(k + z));
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint4 t0, t1, t2;
                        if (r >= len) x[z] = make_uint4(0, 0, 0, 0);
                        split8<false>(x[z], wt, t0, t1, t2);
                        ptx::sts128(bt + group_at(k + z), t0);
                        ptx::sts128(at + group_at(k + z), t1);
                    }
                }
            } else if (need) {
                // two groups a step: their loads in flight together, and a body that fits the instruction cache
#pragma unroll 1
                for (int k = 0; k < BG; k += 2) {
                    uint4 x[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) x[z] = ptx::lds128(bt + group_at(k + z));
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint4 t0, t1, t2;
                        if (r >= len) x[z] = make_uint4(0, 0, 0, 0);
                        split8<true>(x[z], wt, t0, t1, t2);
                        ptx::sts128(bt + group_at(k + z), t0);
                        ptx::sts128(at + group_at(k + z), t1);
                        ptx::sts128(sb + L::X + group_at(k + z), t2);
                    }
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_b);
            if (need) {
                if (!(ok = wait_state(bar_u, (uint32_t)(nu & 1)))) break;
                ++nu;
                ptx::tc_fence_after();
                if (quad * 32 < DAB) {
#pragma unroll
                    for (int b = 0; b < CPT / 16; ++b) {
                        float v[16];
                        ptx::tmem_ld16(t_u + tl + 16 * b, v);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 16; x += 2) {
                            float *z = S + 16 * b + x;
                            const float2 o = make_float2(z[0], z[1]);
                            const float2 n2 = ptx::fma2(make_float2(dec.x, dec.x), o,
                                                        ptx::fma2(make_float2(dec.y, dec.y), o, make_float2(v[x], v[x + 1])));
                            z[0] = n2.x;
                            z[1] = n2.y;
                        }
                    }
                }
                if (item.is(Item::ENDS) && item.is(Item::WHOLE) && want_last && has) {
                    const int row = state_row(slots, num_slots, item.n, 192);
                    if (row >= 0) {
                        float *dst = y.last + (((long long)row * g.H + h) * DAB + r) * DC + col;
#pragma unroll
                        for (int x = 0; x < CPT; x += 4)
                            store4(dst + x, make_float4(S[x], S[x + 1], S[x + 2], S[x + 3]));
                    }
                }
            }
            ++n;
        }
        if (!ok && lane == 0) flag_status(KDA_DEV_WAIT_TIMEOUT);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace la
}  // namespace kda

// ------------------------------------------------------------------ host side

namespace kda {
namespace la {

inline bool tile_map(CUtensorMap *m, const void *x, const Call &c, int d, int tokens = kBox) {
    return kda::tc::make_tmap(m, x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (long long)c.B * c.T, c.H, d, 64,
                              CU_TENSOR_MAP_SWIZZLE_128B, tokens);
}

template <int DB, int DC>
cudaError_t launch_sum(const Geo &g, const SumArgs &a, int roles, const Call &c) {
    constexpr int smem = SumSmem<DB, DC>::ALLOC;
    auto kern = la_sum_kernel<DB, DC>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<dim3(g.W, roles), kSumThreads, smem, c.st>>>(a, g, c.log_decay);
    return cudaGetLastError();
}

// after: behind another kernel of the call
template <int DAB, int DC>
cudaError_t launch_walk(const Geo &g, const WalkArgs &a, int roles, const Call &c, bool after) {
    constexpr int smem = WalkSmem<DAB, DC>::ALLOC;
    auto kern = la_walk_kernel<DAB, DC>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (after)
        return launch_after(kern, g.W * roles, kWalkThreads, smem, c.st, a, g, c.log_decay, c.slots, c.num_slots, roles);
    kern<<<g.W * roles, kWalkThreads, smem, c.st>>>(a, g, c.log_decay, c.slots, c.num_slots, roles);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t tc_forward(const Call &c, const void *q, const void *k, const void *v, const float *s0, void *o,
                       float *last, float *ws) {
    const Geo g = geo_of<kC>(c, 1, 1, true);
    CUtensorMap tq, tk, tv, to;
    if (!tile_map(&tq, q, c, DK) || !tile_map(&tk, k, c, DK) || !tile_map(&tv, v, c, DV) ||
        !tile_map(&to, o, c, DV, kOutBox))
        return cudaErrorInvalidValue;
    Carry y = carry_at(ws, g.W, DK * DV);
    y.s0 = s0;
    y.last = last;
    // a pool is read and written by different CTAs of the walk: it reads cut sequences' states from a copy
    if (c.slots) y.s0_copy = ws + (size_t)3 * g.W * DK * DV;
    cudaError_t e;
    const bool cut = cuts<kC>(g);
    if (cut) {
        SumArgs a{};
        a.role[0] = SumRole{tk, tv, y.sum_in, y.sum_out, 1, 1, last != nullptr};
        if ((e = launch_sum<DK, DV>(g, a, 1, c)) != cudaSuccess) return e;
        if ((e = launch_join<kC>(g, c, DK * DV, true, y, 1)) != cudaSuccess) return e;
    } else if ((e = launch_empty<kC>(g, y, c, DK * DV, false)) != cudaSuccess) {
        return e;
    }
    WalkArgs a{};
    a.role[0] = WalkRole{tq, tk, tv, to, (__nv_bfloat16 *)o, y, 1, 1, 0};
    return launch_walk<DK, DV>(g, a, 1, c, cut);
}

template <int DK, int DV>
cudaError_t tc_backward(const Call &c, const void *q, const void *k, const void *v, const void *d_o, const float *s0,
                        const float *dlast, void *dq, void *dk, void *dv, float *dinit, float *ws) {
    const Geo g = geo_of<kC>(c, 3, 2, true);
    constexpr int E = DK * DV;
    CUtensorMap tq, tk, tv, td, odq, odk, odv;
    if (!tile_map(&tq, q, c, DK) || !tile_map(&tk, k, c, DK) || !tile_map(&tv, v, c, DV) || !tile_map(&td, d_o, c, DV) ||
        !tile_map(&odq, dq, c, DK, kOutBox) || !tile_map(&odk, dk, c, DK, kOutBox) || !tile_map(&odv, dv, c, DV, kOutBox))
        return cudaErrorInvalidValue;
    Carry fwd = carry_at(ws, g.W, E), bwd = carry_at(ws + (size_t)3 * g.W * E, g.W, E);
    fwd.s0 = s0;
    bwd.s0 = dlast;
    bwd.last = dinit;
    cudaError_t e;
    const bool cut = cuts<kC>(g);
    if (cut) {
        SumArgs a{};
        a.role[0] = SumRole{tk, tv, fwd.sum_in, fwd.sum_out, 1, 0, 0};
        a.role[1] = SumRole{tq, td, bwd.sum_in, bwd.sum_out, -1, 1, dinit != nullptr};
        if ((e = launch_sum<DK, DV>(g, a, 2, c)) != cudaSuccess) return e;
        if ((e = launch_join<kC>(g, c, E, true, fwd, 1, &bwd)) != cudaSuccess) return e;
    } else if ((e = launch_empty<kC>(g, bwd, c, E, false)) != cudaSuccess) {
        return e;
    }
    Carry bwd_t = bwd;
    bwd_t.last = nullptr;
    const WalkRole r_dq{td, tv, tk, odq, (__nv_bfloat16 *)dq, fwd, 1, 0, 1}, r_dk{tv, td, tq, odk, (__nv_bfloat16 *)dk, bwd_t, -1, 0, 1},
        r_dv{tk, tq, td, odv, (__nv_bfloat16 *)dv, bwd, -1, 1, 0};
    WalkArgs a{};
    a.role[0] = r_dq;
    a.role[1] = r_dk;
    if (DK == DV) {   // one launch: the three walks of a span share tiles
        a.role[2] = r_dv;
        return launch_walk<DK, DV>(g, a, 3, c, cut);
    }
    if ((e = launch_walk<DV, DK>(g, a, 2, c, cut)) != cudaSuccess) return e;
    a.role[0] = r_dv;
    return launch_walk<DK, DV>(g, a, 1, c, true);
}

}  // namespace la
}  // namespace kda

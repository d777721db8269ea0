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
// read) elsewhere.
#pragma once

#include "kda_chunk_tc.cuh"
#include "kda_la.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace la {

constexpr int kC = 128;                  // tokens of a chunk
constexpr int kBox = 64;                 // token rows of a TMA box
constexpr int kSumThreads = 320;         // producer warp, MMA warp, eight compute warps
constexpr int kWalkThreads = 448;        // producer, MMA, four output warps, eight state warps

// Waits are bounded, and a warp gives up as a whole.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, kda::tc::WAIT_LIMIT_CYCLES));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// 16-byte group g of row r in a 128-byte-swizzled atom (64 bf16 wide)
__device__ __forceinline__ uint32_t swz(int r, int g) { return (uint32_t)(r * 128 + ((g ^ (r & 7)) << 4)); }

// Eight weighted elements as bf16 terms: w x = t0 + t1 (+ t2), each the rounding of what is left.
template <bool THREE>
__device__ __forceinline__ void split8(const uint4 &x, float w, uint4 &t0, uint4 &t1, uint4 &t2) {
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t o0[4], o1[4], o2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = lo_bf16(in[i]) * w, b = hi_bf16(in[i]) * w;
        o0[i] = pack2(a, b);
        const float a1 = a - lo_bf16(o0[i]), b1 = b - hi_bf16(o0[i]);
        o1[i] = pack2(a1, b1);
        o2[i] = THREE ? pack2(a1 - lo_bf16(o1[i]), b1 - hi_bf16(o1[i])) : 0u;
    }
    t0 = make_uint4(o0[0], o0[1], o0[2], o0[3]);
    t1 = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    t2 = make_uint4(o2[0], o2[1], o2[2], o2[3]);
}

// ------------------------------------------------------------------ first pass

// The sum of b c^T over the part of a sequence that lies in a span and goes on behind it
// (in walking order): sum_out, or sum_in when the sequence came from the span before.
// Only the sequence at the span's far edge can have such a part, and its tokens are
// contiguous: the CTA runs over them in tiles of 64 from the far edge towards the near
// one, against the walk, so that what the walk reads first is what L2 saw last.
//
// A tile's three-term products leave TMEM after 12 K steps and are added in fp32 registers,
// scaled by the decay of the tokens behind the tile, so that neither the tensor core's
// accumulation nor a product of many decays costs fp32 accuracy over long sequences.
struct SumRole {
    CUtensorMap b, c;
    float *sum_in, *sum_out;
    int dir;
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
    static constexpr int BYTES = BAR + 8 * (2 * NST + 2 + 1) + 16;
    static constexpr int ALLOC = BYTES + 1024;
    static_assert(ALLOC <= 232448, "shared memory");
};

template <int DB, int DC>
__global__ void __launch_bounds__(kSumThreads, 1)
la_sum_kernel(const __grid_constant__ SumArgs args, Geo g, const float *__restrict__ log_decay) {
    using L = SumSmem<DB, DC>;
    constexpr int NST = L::NST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = ptx::smem_u32(sm);
    const uint32_t bar_full = sb + L::BAR, bar_done = bar_full + 8 * NST, bar_ready = bar_done + 8 * NST,
                   bar_fin = bar_ready + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::BAR + 8 * (2 * NST + 3));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SumRole &role = args.role[blockIdx.y];
    const int dir = role.dir, w = blockIdx.x;
    const long long lo = g.lo(w), hi = g.hi(w), edge = dir > 0 ? hi - 1 : lo;
    Cursor<kC> cur;
    cur.seek(g, edge);
    if (!cur.valid || cur.c == (dir > 0 ? cur.nck - 1 : 0)) return;   // nothing goes on behind the span
    // the part's tokens [ta, tb); did its sequence come from the span before?
    const long long u_near = dir > 0 ? edge - cur.c : edge + (cur.nck - 1 - cur.c);
    const bool through = dir > 0 ? u_near < lo : u_near >= hi;
    const long long near = through ? (dir > 0 ? lo : hi - 1) : u_near;
    const long long ta = dir > 0 ? cur.tok() - (edge - near) * kC : cur.tok();
    const long long tb = dir > 0 ? cur.tok() + kC : min(cur.t1, cur.tok() + (near - edge + 1) * kC);
    const int nt = (int)((tb - ta + kBox - 1) / kBox);
    // tile x counts from the far edge; only a sequence's last tile can be shorter than 64
    auto tile_tok = [&](int x) { return ta + (long long)(dir > 0 ? nt - 1 - x : x) * kBox; };

    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tslot), 256);
        ptx::tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_done + 8 * s, 1);
        }
        ptx::mbar_init(bar_ready, 8);
        ptx::mbar_init(bar_ready + 8, 8);
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
                const int t = (int)tile_tok(n);
                ptx::mbar_arrive_expect_tx(bar, L::STAGE);
#pragma unroll
                for (int a = 0; a < DB / 64; ++a) ptx::tma_load_3d(dst + a * 8192, &role.b, bar, a * 64, cur.h, t);
#pragma unroll
                for (int a = 0; a < DC / 64; ++a)
                    ptx::tma_load_3d(dst + L::BT + a * 8192, &role.c, bar, a * 64, cur.h, t);
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
                 wait_warp(bar_ready + 8 * e, (uint32_t)((n >> 1) & 1));
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t bt = sb + s * L::STAGE;
#pragma unroll
                for (int p = 0; p < 3; ++p) {
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
    } else {
        // ---------------- compute: split the weighted rows; thread <-> state row, half of its columns
        constexpr int CPT = DC / 2;
        const int ct = tid - 64, quad = warp & 3, half = (warp - 2) >> 2;
        const int jr = ct & 63, jq = ct >> 6;     // split: token row, quarter of the columns
        const int row = quad * 32 + lane, col = half * CPT;
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16) + col;
        float S[CPT];
#pragma unroll
        for (int x = 0; x < CPT; ++x) S[x] = 0.f;
        const double lg = (double)log_decay[cur.h];
        const double full_dec = exp(lg * kBox);
        const float full_wt = (float)exp(lg * (dir > 0 ? kBox - 1 - jr : jr + 1));
        double behind = 1.0;         // decay of the tokens behind the tile
        float scale[2];              // the same for the two tiles in flight
        auto drain = [&](int x) {    // adds tile x's sum
            if (!(ok = wait_warp(bar_done + 8 * (x % NST), (uint32_t)((x / NST) & 1)))) return;
            ptx::tc_fence_after();
            if (quad * 32 < DB) {
                const uint32_t u = tl + (x & 1) * 128;
                const float sc = x & 1 ? scale[1] : scale[0];
#pragma unroll
                for (int k = 0; k < CPT / 32; ++k) {
                    float v[32];
                    ptx::tmem_ld32(u + 32 * k, v);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[32 * k + i] = fmaf(sc, v[i], S[32 * k + i]);
                }
            }
        };
        for (int n = 0; n < nt; ++n) {
            const int s = n % NST, e = n & 1;
            // the middle and low terms' buffer is free: tile n - 2 was drained
            if (!(ok = wait_warp(bar_full + 8 * s, (uint32_t)((n / NST) & 1)))) break;
            const int len = (int)min((long long)kBox, tb - tile_tok(n));
            uint8_t *bt = sm + s * L::STAGE, *c0 = bt + L::BT;
            uint8_t *c1 = sm + L::E + e * 2 * L::CT, *c2 = c1 + L::CT;
            const bool live = jr < len;
            // forwards a part ends with a full chunk; backwards the weight counts from the tile's start
            const float wt = full_wt;
#pragma unroll
            for (int k = 0; k < DC / 32; ++k) {
                const int cg = jq * (DC / 32) + k;   // 16-byte group of the row
                const uint32_t at = (cg >> 3) * 8192 + swz(jr, cg & 7);
                uint4 t0 = make_uint4(0, 0, 0, 0), t1 = t0, t2 = t0;   // rows behind the end may hold anything
                if (live) split8<true>(*reinterpret_cast<const uint4 *>(c0 + at), wt, t0, t1, t2);
                *reinterpret_cast<uint4 *>(c0 + at) = t0;
                *reinterpret_cast<uint4 *>(c1 + at) = t1;
                *reinterpret_cast<uint4 *>(c2 + at) = t2;
            }
            if (!live)
#pragma unroll
                for (int k = 0; k < DB / 32; ++k) {
                    const int cg = jq * (DB / 32) + k;
                    *reinterpret_cast<uint4 *>(bt + (cg >> 3) * 8192 + swz(jr, cg & 7)) = make_uint4(0, 0, 0, 0);
                }
            if (e) scale[1] = (float)behind;
            else scale[0] = (float)behind;
            behind *= full_dec;
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_ready + 8 * e);
            if (n > 0) drain(n - 1);   // the tile before, while this one multiplies
            if (!ok) break;
        }
        if (ok) drain(nt - 1);
        if (ok && row < DB) {
            float *dst = (through ? role.sum_in : role.sum_out) + ((long long)w * DB + row) * DC + col;
#pragma unroll
            for (int x = 0; x < CPT; x += 4) store4(dst + x, make_float4(S[x], S[x + 1], S[x + 2], S[x + 3]));
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
    bool fresh;

    __device__ __forceinline__ SpanWalk(const Geo &g, int w, int dir_) : lo(g.lo(w)), hi(g.hi(w)), i(-1), dir(dir_) {
        cur.valid = false;
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
            fresh = false;
            return true;
        }
        return false;
    }
    // items of the sequence behind this one lie in the span too, all of them or some
    __device__ __forceinline__ int left() const { return dir > 0 ? cur.nck - 1 - cur.c : cur.c; }
    __device__ __forceinline__ bool whole_tail() const { return left() < hi - lo - i; }
    __device__ __forceinline__ bool part_over() const { return ends || i == hi - lo - 1; }
};

struct WalkRole {
    CUtensorMap a, b, c;
    __nv_bfloat16 *out;
    Carry y;
    int dir;
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
    static constexpr int BYTES = BAR + 8 * (2 * NST + 9) + 16;
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
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = ptx::smem_u32(sm);
    const uint32_t bar_full = sb + L::BAR, bar_free = bar_full + 8 * NST, bar_sc = bar_free + 8 * NST,
                   bar_in = bar_sc + 8, bar_p = bar_in + 8, bar_b = bar_p + 8, bar_u = bar_b + 8, bar_o = bar_u + 8,
                   bar_x = bar_o + 8, bar_od = bar_x + 8, bar_fin = bar_od + 8;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::BAR + 8 * (2 * NST + 9));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the roles of one span run side by side: they share most of their tiles in L2
    const WalkRole &role = args.role[blockIdx.x % roles];
    const int dir = role.dir, w = blockIdx.x / roles;
    const Carry &y = role.y;
    const bool want_last = y.last != nullptr;

    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tslot), 512);
        ptx::tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_free + 8 * s, 1);
        }
        ptx::mbar_init(bar_sc, 1);
        ptx::mbar_init(bar_in, 1);
        ptx::mbar_init(bar_p, 4);
        ptx::mbar_init(bar_b, 8);
        ptx::mbar_init(bar_u, 1);
        ptx::mbar_init(bar_o, 1);
        ptx::mbar_init(bar_x, 8);
        ptx::mbar_init(bar_od, 4);
        ptx::mbar_init(bar_fin, 1);
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tslot;
    const uint32_t t_sc = tmem, t_oa = tmem + 128, t_oi = tmem + 256, t_u = tmem + 384;
    SpanWalk it(g, w, dir);
    bool ok = true;
    int n = 0;   // chunks so far

    if (warp == 0) {
        // ---------------- producer
        while (it.next(g)) {
            const int s = n % NST;
            if (n >= NST && !(ok = wait_warp(bar_free + 8 * s, (uint32_t)((n / NST - 1) & 1)))) break;
            if (lane == 0) {
                const uint32_t bar = bar_full + 8 * s, dst = sb + L::ST0 + s * L::STAGE;
                const int len = it.cur.len(), t = (int)it.cur.tok(), h = it.cur.h;
                const int boxes = len > kBox ? 2 : 1;
                ptx::mbar_arrive_expect_tx(bar, (uint32_t)(L::STAGE / 2 * boxes));
                for (int x = 0; x < boxes; ++x) {
#pragma unroll
                    for (int a = 0; a < DAB / 64; ++a) {
                        const uint32_t at = dst + a * 16384 + x * 8192;
                        ptx::tma_load_3d(at, &role.a, bar, a * 64, h, t + x * kBox);
                        ptx::tma_load_3d(at + L::AT, &role.b, bar, a * 64, h, t + x * kBox);
                    }
#pragma unroll
                    for (int a = 0; a < DC / 64; ++a)
                        ptx::tma_load_3d(dst + 2 * L::AT + a * 16384 + x * 8192, &role.c, bar, a * 64, h, t + x * kBox);
                }
            }
            __syncwarp();
            ++n;
        }
        if (!ok) {
            if (lane == 0) flag_status(KDA_DEV_WAIT_TIMEOUT);
            for (int k = max(0, n - NST); k < n; ++k)   // copies in flight
                wait_warp(bar_full + 8 * (k % NST), (uint32_t)((k / NST) & 1));
        }
    } else if (warp == 1) {
        // ---------------- MMA
        constexpr uint32_t id_sc = ptx::idesc_bf16_f32(128, 128), id_in = ptx::idesc_bf16_f32(128, DC, false, true),
                           id_u = ptx::idesc_bf16_f32(128, DC, true, true);
        while (it.next(g)) {
            const int s = n % NST;
            const uint32_t at = sb + L::ST0 + s * L::STAGE, bt = at + L::AT, ct = bt + L::AT, ph = (uint32_t)(n & 1);
            // scores: the region is free once the chunk before has multiplied its P
            ok = wait_warp(bar_full + 8 * s, (uint32_t)((n / NST) & 1)) && (n == 0 || wait_warp(bar_o, ph ^ 1u));
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < DAB / 16; ++ks)
                    ptx::mma_bf16(t_sc, kda::tc::kdesc(at, ks, kC), kda::tc::kdesc(bt, ks, kC), id_sc, ks > 0);
                ptx::mma_commit(bar_sc);
            }
            __syncwarp();
            ok = wait_warp(bar_x, ph) && (n == 0 || wait_warp(bar_od, ph ^ 1u));
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < DAB / 16; ++ks)
                    ptx::mma_bf16(t_oi, kda::tc::kdesc(at, ks, kC),
                                  ptx::desc_mnmajor_sw128(sb + L::X + ks * 2048, DAB * 128, 1024), id_in, ks > 0);
                ptx::mma_commit(bar_in);
            }
            __syncwarp();
            if (!(ok = wait_warp(bar_b, ph))) break;
            ptx::tc_fence_after();
            if (!it.part_over() || (it.ends && want_last)) {
                if (lane == 0) {
                    auto term = [&](uint32_t x, uint32_t acc) {
#pragma unroll
                        for (int ks = 0; ks < kC / 16; ++ks)
                            ptx::mma_bf16(t_u, ptx::desc_mnmajor_sw128(x + ks * 2048, 16384, 1024),
                                          ptx::desc_mnmajor_sw128(ct + ks * 2048, 16384, 1024), id_u, acc + ks > 0);
                    };
                    // small terms first: the accumulator is least rounded while it is small
                    if (want_last) term(sb + L::X, 0);
                    term(at, want_last ? 1 : 0);
                    term(bt, 1);
                    ptx::mma_commit(bar_u);
                }
                __syncwarp();
            }
            if (!(ok = wait_warp(bar_p, ph))) break;
            ptx::tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < kC / 16; ++ks)
                    ptx::mma_bf16_ts(t_oa, t_sc + ks * 8, ptx::desc_mnmajor_sw128(ct + ks * 2048, 16384, 1024), id_in,
                                     ks > 0);
                ptx::mma_commit(bar_o);
                ptx::mma_commit(bar_free + 8 * s);
            }
            __syncwarp();
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
        const uint32_t tl = (uint32_t)(quad * 32) << 16;
        float step[16];   // g^(15 - m) forwards, g^m backwards, m = 0..15
        float l2 = 0.f;   // log2 g: P and out are rounded to bf16, which a fast exponential's error does not reach
        int head = -1;
        while (it.next(g)) {
            const uint32_t ph = (uint32_t)(n & 1);
            const int h = it.cur.h, len = it.cur.len();
            const long long t = it.cur.tok();
            if (h != head) {
                head = h;
                l2 = log_decay[h] * 1.44269504f;
#pragma unroll
                for (int m = 0; m < 16; ++m) step[m] = kda::tc::exp2_fast(l2 * (dir > 0 ? 15 - m : m));
            }
            if (!(ok = wait_warp(bar_sc, ph))) break;
            ptx::tc_fence_after();
            // 32 score columns a step.  In a 16-column block all on one side of the diagonal
            // g^|i-j| = g^(distance to its nearest column) step[m]; on the diagonal each has its own.
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t p[16];
                if (dir > 0 ? b > quad : b < quad) {
#pragma unroll
                    for (int x = 0; x < 16; ++x) p[x] = 0u;
                } else {
                    float s[32];
                    ptx::tmem_ld32(t_sc + tl + 32 * b, s);
                    ptx::tmem_wait_ld();
                    if (b != quad) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int j0 = 32 * b + 16 * k;
                            const float r = kda::tc::exp2_fast(l2 * (dir > 0 ? i - j0 - 15 : j0 - i));
#pragma unroll
                            for (int m = 0; m < 16; ++m) s[16 * k + m] *= r * step[m];
                        }
                    } else {
#pragma unroll
                        for (int m = 0; m < 32; ++m) {
                            const int d = (lane - m) * dir;
                            s[m] = d >= 0 ? s[m] * kda::tc::exp2_fast(l2 * d) : 0.f;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 16; ++x) p[x] = pack2(s[2 * x], s[2 * x + 1]);
                    if (dir < 0 && 32 * b + 32 > len) {
                        // backwards in time the masked side does not cover the rows behind the end
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const int j = 32 * b + 2 * x;
                            if (j >= len) p[x] = 0u;
                            else if (j + 1 >= len) p[x] &= 0xffffu;
                        }
                    }
                }
                ptx::tmem_st16(t_sc + tl + 16 * b, p);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_p);
            if (!(ok = wait_warp(bar_o, ph))) break;
            ptx::tc_fence_after();
            const float up = i < len ? kda::tc::exp2_fast(l2 * (dir > 0 ? i + 1 : len - 1 - i)) : 0.f;
            __nv_bfloat16 *dst = role.out + ((t + i) * g.H + h) * DC;
#pragma unroll
            for (int b = 0; b < DC / 16; ++b) {
                float oa[16], oi[16];
                ptx::tmem_ld16(t_oa + tl + 16 * b, oa);
                ptx::tmem_ld16(t_oi + tl + 16 * b, oi);
                ptx::tmem_wait_ld();
                if (i < len) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t r[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            r[k] = pack2(fmaf(up, oi[8 * x + 2 * k], oa[8 * x + 2 * k]),
                                         fmaf(up, oi[8 * x + 2 * k + 1], oa[8 * x + 2 * k + 1]));
                        *reinterpret_cast<uint4 *>(dst + 16 * b + 8 * x) = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_od);
            ++n;
        }
        if (!ok && lane == 0) flag_status(KDA_DEV_WAIT_TIMEOUT);
    } else {
        // ---------------- state.  Thread <-> state row, and <-> token row when it weighs b; half the columns.
        constexpr int CPT = DC / 2, BG = DAB / 16;   // state columns, 16-byte groups of a b row
        const int quad = warp & 3, half = (warp - 6) >> 2, r = quad * 32 + lane, col = half * CPT;
        const uint32_t tl = ((uint32_t)(quad * 32) << 16) + col;
        const bool has = r < DAB;
        float S[CPT];
        int head = -1, wlen = -1, nu = 0;
        float wt = 0.f;                          // this token row's weight
        float2 dec = make_float2(0.f, 0.f);      // decay of the chunk
        while (it.next(g)) {
            const uint32_t ph = (uint32_t)(n & 1);
            const int s = n % NST, h = it.cur.h, len = it.cur.len();
            if (h != head || len != wlen) {
                head = h;
                wlen = len;
                const float lg = log_decay[h];
                wt = r < len ? (float)exp((double)lg * (dir > 0 ? len - 1 - r : r + 1)) : 0.f;
                dec = decay2(lg, len);
            }
            if (it.first) {
                const float *src = nullptr;
                const int row = state_row(slots, num_slots, it.cur.n);
                if (it.from_before) src = y.start + (long long)w * DAB * DC;
                else if (y.s0_copy && !it.whole_tail()) src = y.s0_copy + ((long long)it.cur.n * g.H + h) * (DAB * DC);
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
                    *reinterpret_cast<uint4 *>(sm + L::X + (cg >> 3) * (DAB * 128) + swz(r, cg & 7)) =
                        make_uint4(pack2(S[8 * k], S[8 * k + 1]), pack2(S[8 * k + 2], S[8 * k + 3]),
                                   pack2(S[8 * k + 4], S[8 * k + 5]), pack2(S[8 * k + 6], S[8 * k + 7]));
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_x);
            uint8_t *at = sm + L::ST0 + s * L::STAGE, *bt = at + L::AT, *ct = bt + L::AT;
            if (!(ok = wait_warp(bar_full + 8 * s, (uint32_t)((n / NST) & 1)))) break;
            if (r >= len) {   // what lies behind the end may be another sequence's, or anything
#pragma unroll
                for (int k = 0; k < CPT / 8; ++k) {
                    const int cg = col / 8 + k;
                    *reinterpret_cast<uint4 *>(ct + (cg >> 3) * 16384 + swz(r, cg & 7)) = make_uint4(0, 0, 0, 0);
                }
            }
            // inter done: scores are taken too, the tiles of A and X are free
            if (!(ok = wait_warp(bar_in, ph))) break;
            const bool need = !it.part_over() || (it.ends && want_last);
            if (need) {
#pragma unroll
                for (int k = 0; k < BG; ++k) {
                    const int cg = half * BG + k;
                    const uint32_t off = (cg >> 3) * 16384 + swz(r, cg & 7);
                    uint4 t0 = make_uint4(0, 0, 0, 0), t1 = t0, t2 = t0;
                    if (r < len) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(bt + off);
                        if (want_last) split8<true>(x, wt, t0, t1, t2);
                        else split8<false>(x, wt, t0, t1, t2);
                    }
                    *reinterpret_cast<uint4 *>(bt + off) = t0;
                    *reinterpret_cast<uint4 *>(at + off) = t1;
                    if (want_last) *reinterpret_cast<uint4 *>(sm + L::X + off) = t2;
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_b);
            if (need) {
                if (!(ok = wait_warp(bar_u, (uint32_t)(nu & 1)))) break;
                ++nu;
                ptx::tc_fence_after();
                if (quad * 32 < DAB) {
#pragma unroll
                    for (int b = 0; b < CPT / 16; ++b) {
                        float v[16];
                        ptx::tmem_ld16(t_u + tl + 16 * b, v);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            float &z = S[16 * b + x];
                            z = fmaf(dec.x, z, fmaf(dec.y, z, v[x]));
                        }
                    }
                }
                if (it.ends && want_last && has) {
                    const int row = state_row(slots, num_slots, it.cur.n);
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

inline bool tile_map(CUtensorMap *m, const void *x, const Call &c, int d) {
    return kda::tc::make_tmap(m, x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (long long)c.B * c.T, c.H, d, 64,
                              CU_TENSOR_MAP_SWIZZLE_128B);
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

template <int DAB, int DC>
cudaError_t launch_walk(const Geo &g, const WalkArgs &a, int roles, const Call &c) {
    constexpr int smem = WalkSmem<DAB, DC>::ALLOC;
    auto kern = la_walk_kernel<DAB, DC>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<g.W * roles, kWalkThreads, smem, c.st>>>(a, g, c.log_decay, c.slots, c.num_slots, roles);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t tc_forward(const Call &c, const void *q, const void *k, const void *v, const float *s0, void *o,
                       float *last, float *ws) {
    const Geo g = geo_of<kC>(c);
    CUtensorMap tq, tk, tv;
    if (!tile_map(&tq, q, c, DK) || !tile_map(&tk, k, c, DK) || !tile_map(&tv, v, c, DV))
        return cudaErrorInvalidValue;
    Carry y = carry_at(ws, g.W, DK * DV);
    y.s0 = s0;
    y.last = last;
    // a pool is read and written by different CTAs of the walk: it reads cut sequences' states from a copy
    if (c.slots) y.s0_copy = ws + (size_t)3 * g.W * DK * DV;
    cudaError_t e;
    if (cuts<kC>(g)) {
        SumArgs a{};
        a.role[0] = SumRole{tk, tv, y.sum_in, y.sum_out, 1};
        if ((e = launch_sum<DK, DV>(g, a, 1, c)) != cudaSuccess) return e;
        if ((e = launch_join<kC, 1>(g, y, c, DK * DV)) != cudaSuccess) return e;
    }
    WalkArgs a{};
    a.role[0] = WalkRole{tq, tk, tv, (__nv_bfloat16 *)o, y, 1, 0};
    return launch_walk<DK, DV>(g, a, 1, c);
}

template <int DK, int DV>
cudaError_t tc_backward(const Call &c, const void *q, const void *k, const void *v, const void *d_o, const float *s0,
                        const float *dlast, void *dq, void *dk, void *dv, float *dinit, float *ws) {
    const Geo g = geo_of<kC>(c);
    constexpr int E = DK * DV;
    CUtensorMap tq, tk, tv, td;
    if (!tile_map(&tq, q, c, DK) || !tile_map(&tk, k, c, DK) || !tile_map(&tv, v, c, DV) || !tile_map(&td, d_o, c, DV))
        return cudaErrorInvalidValue;
    Carry fwd = carry_at(ws, g.W, E), bwd = carry_at(ws + (size_t)3 * g.W * E, g.W, E);
    fwd.s0 = s0;
    bwd.s0 = dlast;
    bwd.last = dinit;
    cudaError_t e;
    if (cuts<kC>(g)) {
        SumArgs a{};
        a.role[0] = SumRole{tk, tv, fwd.sum_in, fwd.sum_out, 1};
        a.role[1] = SumRole{tq, td, bwd.sum_in, bwd.sum_out, -1};
        if ((e = launch_sum<DK, DV>(g, a, 2, c)) != cudaSuccess) return e;
        if ((e = launch_join<kC, 1>(g, fwd, c, E)) != cudaSuccess) return e;
        if ((e = launch_join<kC, -1>(g, bwd, c, E)) != cudaSuccess) return e;
    }
    Carry bwd_t = bwd;
    bwd_t.last = nullptr;
    const WalkRole r_dq{td, tv, tk, (__nv_bfloat16 *)dq, fwd, 1, 1}, r_dk{tv, td, tq, (__nv_bfloat16 *)dk, bwd_t, -1, 1},
        r_dv{tk, tq, td, (__nv_bfloat16 *)dv, bwd, -1, 0};
    WalkArgs a{};
    a.role[0] = r_dq;
    a.role[1] = r_dk;
    if (DK == DV) {   // one launch: the three walks of a span share tiles
        a.role[2] = r_dv;
        return launch_walk<DK, DV>(g, a, 3, c);
    }
    if ((e = launch_walk<DV, DK>(g, a, 2, c)) != cudaSuccess) return e;
    a.role[0] = r_dv;
    return launch_walk<DK, DV>(g, a, 1, c);
}

}  // namespace la
}  // namespace kda

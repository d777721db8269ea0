// Linear attention with a decay for each head: what its kernels share.
//
// Per (sequence, head), with g = exp(log_decay_h), one constant rate per head:
//   S_t = g S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t                       (S: dk x dv, fp32)
// A chunk of L tokens that starts from state S (0-based i, j):
//   o_i = g^{i+1} S^T q_i + sum_{j<=i} g^{i-j} (q_i . k_j) v_j
//   S'  = g^L S + sum_j g^{L-1-j} k_j v_j^T
// The backward pass has the same form.  With X = g (adjoint of the state at the next
// chunk's first token), and X = dL/dfinal_state behind the last token:
//   dq_i = g^{i+1} S do_i       + sum_{j<=i} g^{i-j} (do_i . v_j) k_j
//   dk_i = g^{L-1-i} X v_i      + sum_{j>=i} g^{j-i} (v_i . do_j) q_j
//   dv_i = g^{L-1-i} X^T k_i    + sum_{j>=i} g^{j-i} (k_i . q_j) do_j
//   X'   = g^L X + sum_j g^{j+1} q_j do_j^T,   dL/dinit_state = X at the first token
// So one walk, in either direction, computes all of them: rows a attend to rows b
// and sum rows c, out_i = u_i S^T a_i + sum_j g^|i-j| (a_i . b_j) c_j with the state
// summing b c^T:
//   forward (a, b, c) = (q, k, v);  dq (do, v, k) on S^T;  backwards in time
//   dk (v, do, q) on X^T and dv (k, q, do) on X.
//
// Work split: the (head, chunk) items of a call are laid out head by head and cut
// into W equal spans, one per CTA, so that every SM gets the same share whatever the
// lengths.  A span may start or end inside a sequence; a first pass sums b c^T over
// the part of each cut sequence that lies in a span, a small scan joins those sums
// into the state every span starts from, and the walk then runs each span from there.
#pragma once

#include <algorithm>

#include "kda_common.cuh"

namespace kda {
namespace la {

constexpr int kSMs = 148;

// Token geometry of one call.  Chunks of C tokens are counted from each sequence's
// start; chunk c of sequence n has slot f(n) + c, f(n) = floor(t0 / C) + n for packed
// input (unique, below floor(T / C) + N, with holes) and n ceil(T / C) for a dense batch.
struct Geo {
    const int32_t *cu;   // packed offsets, or null
    int T, N, H;         // tokens of a row (packed: of the call), sequences, heads
    int nslots;          // chunk slots of one head
    int W;               // spans: `rem` of them have (per + 1) unit items, the others per unit
    int rem;
    long long per;
    int unit;            // 1, or the chunks of a sequence: then no sequence is cut
    __host__ __device__ long long items() const { return (long long)H * nslots; }
    __host__ __device__ long long lo(int w) const { return unit * (w * per + (w < rem ? w : rem)); }
    __host__ __device__ long long hi(int w) const { return lo(w + 1); }
};

// Where one item lies.  seek and step are warp-collective (all 32 lanes, converged).
template <int C>
struct Cursor {
    long long t0, t1;    // the sequence's tokens
    int h, n, c, nck;    // head, sequence, chunk and number of chunks of the sequence
    int slot;
    bool valid;          // false: a hole between packed sequences

    __device__ __forceinline__ static int first_slot(const Geo &g, int n) {
        return min(max(g.cu[n], 0), g.T) / C + n;
    }

    __device__ __forceinline__ void seek(const Geo &g, long long u) {
        // (a 64-bit division takes a thousand cycles where its instructions are not yet cached)
        h = (u | g.nslots) >> 32 ? (int)(u / g.nslots) : (int)((unsigned)u / (unsigned)g.nslots);
        slot = (int)(u - (long long)h * g.nslots);
        if (!g.cu) {
            nck = (g.T + C - 1) / C;
            n = slot / nck;
            c = slot - n * nck;
            t0 = (long long)n * g.T;
            t1 = t0 + g.T;
            valid = true;
            return;
        }
        // the last sequence whose first slot is not behind this one: a 32-way search
        const int lane = threadIdx.x & 31;
        int a = 0, b = g.N;
        valid = false;
        while (true) {
            const int step = max(1, (b - a + 31) / 32);
            const int m = a + lane * step;
            const unsigned hit = __ballot_sync(0xffffffffu, m < b && first_slot(g, m) <= slot);
            const int cnt = hit == 0xffffffffu ? 32 : __ffs(~hit) - 1;
            if (cnt == 0) return;
            a += (cnt - 1) * step;
            if (step == 1) break;
            b = min(b, a + step);
        }
        n = a;
        seq_span(g.cu, g.T, n, t0, t1);
        c = slot - first_slot(g, n);
        nck = (int)((t1 - t0 + C - 1) / C);
        valid = c >= 0 && c < nck;
    }

    // From the item u - DIR to the item u.
    template <int DIR>
    __device__ __forceinline__ void step(const Geo &g, long long u) {
        if (valid && c + DIR >= 0 && c + DIR < nck) {
            c += DIR;
            slot += DIR;
        } else {
            seek(g, u);
        }
    }
    __device__ __forceinline__ long long tok() const { return t0 + (long long)c * C; }
    __device__ __forceinline__ int len() const { return (int)min((long long)C, t1 - tok()); }
};

// A head's rate.  Below -1e30 every power but the 0th is 0 all the same, and the products with
// distances, also in fp32 and with 1 / log 2, stay finite (an infinite one times a distance of 0 is NaN).
__device__ __forceinline__ float rate_of(const float *log_decay, int h) {
    const float x = log_decay[h];
    return x < -1e30f ? -1e30f : x;
}

// Flags entries of a slot table that are outside the pool: no span visits a packed sequence without
// tokens.  The tensor-core walk calls it with threads that have to wait for their first tiles anyway (not inlined:
// it costs the loops behind it registers; in the fp32 walk it cost 2 % even so, which has a launch of the join for it).
__device__ __noinline__ void check_slots(int seqs, const int32_t *slots, int num_slots, int thread, int threads) {
    for (int n = blockIdx.x * threads + thread; n < seqs; n += gridDim.x * threads)
        if (slots[n] < -1 || slots[n] >= num_slots) flag_status(KDA_DEV_BAD_SLOT);
}

// exp(log_decay e) with the exponent's product in 64 bits, as the sum of two floats:
// a chunk's decay is applied once per chunk of a sequence, so an error in its last
// place would grow with the number of chunks.
__device__ __noinline__ double exp64(double x) { return exp(x); }   // one copy in a kernel
__device__ __forceinline__ float2 decay2(float log_decay, double e) {
    const double x = exp64((double)log_decay * e);
    const float hi = (float)x;
    return make_float2(hi, (float)(x - (double)hi));
}

// One set of states that the spans hand on: sums of the cut parts and start states.
struct Carry {
    float *sum_in;       // [W][dk dv] the part that comes from the span before (in walking order)
    float *sum_out;      // [W][dk dv] the part that starts in the span and goes on behind it
    float *start;        // [W][dk dv] the state at the span's first item
    const float *s0;     // initial states [rows][H][dk dv] or null (zeros)
    float *s0_copy;      // [N][H][dk dv]: s0 as read, kept when `last` overwrites it; or null
    float *last;         // final states [rows][H][dk dv] or null
};

// Joins the cut parts of up to two sets of carried states (blockIdx.z), each in its direction.
// Thread = kJoinVecs x four elements of the state; CTA column w (blockIdx.x < W) follows the
// sequence that goes on behind span w from span to span.  The sums are independent loads,
// fetched kAhead spans ahead of the recurrence that adds them up, and the decays of 32 spans at
// a time are one warp's work (fp64 exponentials by every thread took longer than the loads).
// finals: the part in the span where the sequence ends has a sum too, and `last` is written
// here; without it the walk writes it.  Columns W.. (packed): one sequence each, handed
// through when it has no tokens.
constexpr int kJoinVecs = 2;
struct Join {
    Carry y;
    int dir;
    int finals;
};
struct Joins {
    Join j[2];
};
template <int C>
__global__ void __launch_bounds__(256) la_join_kernel(Geo g, const __grid_constant__ Joins joins,
                                                      const float *__restrict__ log_decay, int E,
                                                      const int32_t *__restrict__ slots, int num_slots) {
    let_next_start();
    const Join &job = joins.j[blockIdx.z];
    const Carry &y = job.y;
    const int dir = job.dir;
    const int e0 = (blockIdx.y * 256 * kJoinVecs + threadIdx.x) * 4;   // and every 1024 on; E is a multiple of 1024 kJoinVecs
    struct V {
        float4 v[kJoinVecs];
    };
    auto load = [&](const float *p) {
        V r;
#pragma unroll
        for (int k = 0; k < kJoinVecs; ++k) r.v[k] = load4(p + e0 + k * 1024);
        return r;
    };
    auto store = [&](float *p, const V &x) {
#pragma unroll
        for (int k = 0; k < kJoinVecs; ++k) store4(p + e0 + k * 1024, x.v[k]);
    };
    V zero;
#pragma unroll
    for (int k = 0; k < kJoinVecs; ++k) zero.v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if ((int)blockIdx.x >= g.W) {
        const int n = blockIdx.x - g.W;
        long long t0, t1;
        seq_span(g.cu, g.T, n, t0, t1);
        const int row = state_row(slots, num_slots, n);
        wait_for_previous();
        if (t1 > t0 || !y.last || y.last == y.s0 || row < 0) return;
        for (int h = 0; h < g.H; ++h) {
            const long long off = ((long long)row * g.H + h) * E;
            store(y.last + off, y.s0 ? load(y.s0 + off) : zero);
        }
        return;
    }
    const int w0 = blockIdx.x;
    const long long lo = g.lo(w0), hi = g.hi(w0);
    Cursor<C> cur;
    const long long edge = dir > 0 ? hi - 1 : lo;
    cur.seek(g, edge);
    // the sequence at the span's far edge must start inside the span and go on behind it
    const long long u_first = dir > 0 ? edge - cur.c : edge + (cur.nck - 1 - cur.c);
    const bool mine = cur.valid && cur.c != (dir > 0 ? cur.nck - 1 : 0) && (dir > 0 ? u_first >= lo : u_first < hi);
    if (!mine) {
        wait_for_previous();
        return;
    }
    const long long u_last = dir > 0 ? u_first + cur.nck - 1 : u_first - (cur.nck - 1);
    const int row = state_row(slots, num_slots, cur.n);
    const long long off = ((long long)max(row, 0) * g.H + cur.h) * E;
    // spans behind w0 that the sequence crosses from edge to edge; in the next one it ends
    auto crossed = [&](int x) { return x >= 0 && x < g.W && (dir > 0 ? u_last >= g.hi(x) : u_last < g.lo(x)); };
    // tokens of the sequence in span x
    auto tokens = [&](int x) -> double {
        if (x == w0) return dir > 0 ? (double)(cur.c + 1) * C : (double)(cur.t1 - cur.tok());
        if (crossed(x)) return (double)(g.hi(x) - g.lo(x)) * C;
        return dir > 0 ? (double)(cur.t1 - (cur.t0 + (g.lo(x) - u_first) * C)) : (double)(g.hi(x) - u_last) * C;
    };
    __shared__ float2 dec[32];   // of the spans from `base` on
    int base = 0;
    auto decays = [&]() {
        __syncthreads();
        if (threadIdx.x < 32) {
            const int x = w0 + (base + (int)threadIdx.x) * dir;
            // behind the span where the sequence ends nothing is asked for
            dec[threadIdx.x] = threadIdx.x + base > 0 && !crossed(x - dir) && x - dir != w0
                                   ? make_float2(0.f, 0.f)
                                   : decay2(rate_of(log_decay, cur.h), tokens(x));
        }
        __syncthreads();
    };
    decays();
    auto add = [](float2 d, const V &s, const V &u) {
        auto one = [&](float a, float b) { return fmaf(d.x, a, fmaf(d.y, a, b)); };
        V r;
#pragma unroll
        for (int k = 0; k < kJoinVecs; ++k)
            r.v[k] = make_float4(one(s.v[k].x, u.v[k].x), one(s.v[k].y, u.v[k].y), one(s.v[k].z, u.v[k].z),
                                 one(s.v[k].w, u.v[k].w));
        return r;
    };
    wait_for_previous();
    const V s0 = row >= 0 && y.s0 ? load(y.s0 + off) : zero;
    const V out0 = load(y.sum_out + (long long)w0 * E);
    constexpr int kAhead = 4;
    V u[kAhead];
    int w = w0 + dir, m = 0;
    auto fetch = [&]() {   // the sums of spans w.. that are crossed
        m = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (m == k && crossed(w + k * dir)) {
                u[k] = load(y.sum_in + (long long)(w + k * dir) * E);
                m = k + 1;
            }
    };
    fetch();
    if (y.s0_copy) store(y.s0_copy + ((long long)cur.n * g.H + cur.h) * E, s0);
    V s = add(dec[0], s0, out0);
    int i = 1;
    store(y.start + (long long)w * E, s);
    while (m > 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k < m) {
                if (i - base == 32) {
                    base = i;
                    decays();
                }
                s = add(dec[i - base], s, u[k]);
                ++i;
                w += dir;
                store(y.start + (long long)w * E, s);
            }
        fetch();
    }
    if (job.finals && y.last && row >= 0) {
        const V end = load(y.sum_in + (long long)w * E);
        if (i - base == 32) {
            base = i;
            decays();
        }
        store(y.last + off, add(dec[i - base], s, end));
    }
}

}  // namespace la
}  // namespace kda

// Gated linear recurrence over packed sequences, per channel:
//     log form      a = exp(max(g, lb)),  h_t = a_t h_{t-1} + x_t
//     sigmoid form  a = sigmoid(g),       h_t = a_t h_{t-1} + (1 - a_t) x_t
// its backward pass and its single token.
//
// 6 bytes an element forward, 10 backward (bf16; 12 in the sigmoid form). Bound by HBM where
// walkers are many, by the instructions of one warp along the longest sequence (41 ns a row)
// where they just fill the GPU: 31744 x 12288 in four sequences 502 us a call (4.7 TB/s); and by
// the second reading where time is cut: 8192 x 2048 backward, sigmoid form, 50 us (4.0 TB/s).
// Each element is read once, decayed once and written once by a walker, which carries the
// states of its channels in registers; seven walkers share an SM, and nothing waits for
// another CTA.
//
// Where channels times sequences are too few to fill the GPU, time is cut too. A run of
// rows is the map c -> A c + H of the state before it (A the product of its a, H its result
// from zero; a sequence's first row drops what came before): a first kernel reduces each
// piece to its map, and the walker of a piece composes the maps of the pieces before it,
// back to where its sequence began, before it starts. That reads two of the tensors a second
// time. A forward whose inputs fit L2 finds them there (8192 x 2048: 7 of 67 MB come from DRAM);
// larger ones do not (131072 x 257 fp32: 273 of 270 MB), nor does the backward, whose second pass
// streams its other tensors over them (8192 x 2048: it reads 117 of 134 MB). Handing states from CTA to CTA inside one kernel would read
// once, but measured slower: links of a chain have to wait for one another, and every row is
// walked twice by the CTA that holds it (31744 x 12288: 768 us; 8192 x 2048 backward: 82
// against 47 then; with flags behind fences a handover alone took 8 us under load). What is
// composed, and in which order, goes by the shapes: results do not depend on timing.
#include <type_traits>

#include "kda_layer.cuh"

namespace kda {

namespace {

// Walkers that run at the same time, with rings of 24 KiB.
constexpr int kWalkerSlots = 148 * 7;
constexpr int kMinPiece = 64;       // rows of a piece, at least
constexpr int kStage = 8;           // rows of a stage
constexpr int ring_stages(int lb, int tensors) { return 96 / lb / tensors; }
// Rows that are unrolled: a stage, or two where a row of single elements takes so many
// instructions that a stage of them would not stay in the instruction cache.
template <int G> constexpr int unrolled() { return G > 2 ? kStage : 2; }
template <typename T, int G, int LB, int N> using ScanRing = Ring<T, G, LB, kStage, N, ring_stages(LB, N)>;

// exp(g) of log-decays that are bf16, on the SFU, whose exponential is that of 2: log2 e is split
// (Cody and Waite) into a head of 16 bits, whose product with the 8 bits of g is exact, and a
// rest, whose factor is 1 + g rest ln 2 but for its square. That is off by 7 2^-24 of a at most:
// 4 by the exponential, 1 by the last rounding, and (g rest ln 2)^2 / 2 < 1.6 where a is a
// normal number. One product with log2 e would add 2 |g| of them, the same way at every
// step of a constant gate. A lower bound of more than 8 bits rounds the product: |bound| more.
constexpr float kLog2eHead = 47274.f / 32768.f;
constexpr float kLog2eRest = (float)((1.4426950408889634 - 47274. / 32768.) * 0.6931471805599453);
// Below it a is 0; and 0 (1 + g rest ln 2) stays 0 for g = -inf.
constexpr float kNoDecayLeft = -150.f;

// a of the gate input, and the weight b of x in the sigmoid form: 1 - a without the
// cancellation, since a is close to 1 where memories are long. lb is -inf without a bound.
// bf16 inputs take the SFU's exponential (in the sigmoid form of a rounded product, off by
// (4 + 2 |g|) 2^-24 of the smaller of a and 1 - a); fp32 inputs take expf.
template <typename T, bool SIG> __device__ __forceinline__ void decay(float g, float lb, float &a, float &b) {
    constexpr bool FAST = sizeof(T) == 2;
    if (SIG) {
        const float e = FAST ? ex2_fast(-kLog2e * fabsf(g)) : expf(-fabsf(g));
        const float r = FAST ? rcp_fast(1.f + e) : 1.f / (1.f + e), q = e * r;
        a = g >= 0.f ? r : q;
        b = g >= 0.f ? q : r;
    } else if (FAST) {
        g = max_nan(g, fmaxf(lb, kNoDecayLeft));
        a = ex2_fast(g * kLog2eHead);
        a = fmaf(a, g * kLog2eRest, a);
        b = 1.f;
    } else {
        a = expf(max_nan(g, lb));
        b = 1.f;
    }
}

// Of a lane's channels in N rows: g becomes a, one operation of all of them after the other
// where the operations are few (see steps_fwd).
template <typename T, bool SIG, int N, int W>
__device__ __forceinline__ void decays(float (&a)[N][W], float lb, float (&b)[N][W]) {
    if constexpr (!SIG && sizeof(T) == 2) {
        float head[W], rest[W], f[N][W];
        vset(head, kLog2eHead);
        vset(rest, kLog2eRest);
        const float least = fmaxf(lb, kNoDecayLeft);
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
            for (int i = 0; i < W; ++i) a[s][i] = max_nan(a[s][i], least);
#pragma unroll
        for (int s = 0; s < N; ++s) vmul(a[s], rest, f[s]);
#pragma unroll
        for (int s = 0; s < N; ++s) vmul(a[s], head, a[s]);
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
            for (int i = 0; i < W; ++i) a[s][i] = ex2_fast(a[s][i]);
#pragma unroll
        for (int s = 0; s < N; ++s) vfma(a[s], f[s], a[s], a[s]);
#pragma unroll
        for (int s = 0; s < N; ++s) vset(b[s], 1.f);
    } else {
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
            for (int i = 0; i < W; ++i) decay<T, SIG>(a[s][i], lb, a[s][i], b[s][i]);
    }
}
template <typename T, bool SIG, int W> __device__ __forceinline__ void decays(const float (&g)[W], float lb, float (&a)[W], float (&b)[W]) {
    float c[1][W], d[1][W];
#pragma unroll
    for (int i = 0; i < W; ++i) c[0][i] = g[i];
    decays<T, SIG, 1>(c, lb, d);
#pragma unroll
    for (int i = 0; i < W; ++i) a[i] = c[0][i], b[i] = d[0][i];
}

// State n's channels, or zeros.
template <int W> __device__ __forceinline__ void get_state(const float *states, int n, int c, int D, float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = states && c + i < D ? states[(long long)n * D + c + i] : 0.f;
}

template <int W> __device__ __forceinline__ void put_state(float *states, int n, int c, int D, const float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i)
        if (c + i < D) states[(long long)n * D + c + i] = v[i];
}

// ---------------------------------------------------------------- pieces
// The rows of a piece.
__device__ __forceinline__ void piece_rows(const ScanCut &cut, const RowSpan &sp, int piece, int &b, int &e) {
    if (cut.kind == kCutBatch) {
        const int n = piece / cut.per, j = piece - n * cut.per;
        b = n * sp.T + j * cut.rows;
        e = n * sp.T + (j + 1 == cut.per ? sp.T : (j + 1) * cut.rows);  // the last piece's rows may end beyond 32 bits
    } else if (cut.kind == kCutSeqs) {
        b = min(max(sp.cu[piece], 0), sp.R);
        e = min(max(sp.cu[piece + 1], b), sp.R);
    } else {
        b = min(piece * cut.rows, sp.R);
        e = piece + 1 == cut.pieces ? sp.R : min(b + cut.rows, sp.R);
    }
}

// The piece that holds a row (of the cuts that carry).
__device__ __forceinline__ int piece_of(const ScanCut &cut, const RowSpan &sp, int row) {
    if (cut.kind == kCutBatch) {
        const int n = row / sp.T;
        return n * cut.per + (row - n * sp.T) / cut.rows;
    }
    return min(row / cut.rows, cut.pieces - 1);
}

// A lane's channels of a piece's map: A and H of each, W pairs side by side. A map where a
// sequence begins leaves nothing of what came before, not even as 0 x inf: its A is below 0.
template <int W> struct __align__(16) Map {
    float2 ch[W];
};

// The map of piece 0 of the lane whose first channel is c; a piece's maps take its channel
// units in full.
template <int W> __device__ __forceinline__ Map<W> *lane_map(const ScanCut &cut, int c) {
    return static_cast<Map<W> *>(cut.maps) + c / W;
}

// c <- the state behind pieces first, first + step, .. before `piece`. at: the lane's map of
// piece 0, `pitch` maps apart from the next piece's.
template <int W>
__device__ __forceinline__ void compose(const Map<W> *at, long long pitch, int first, int piece, int step, float (&c)[W]) {
    vset(c, 0.f);
    constexpr int BATCH = 8;  // loads in flight
    for (int k = first; k != piece;) {
        Map<W> m[BATCH];
        const int n = min(BATCH, (piece - k) * step);
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
            if (u < n) {
                const float4 *q = reinterpret_cast<const float4 *>(at + (long long)(k + u * step) * pitch);
#pragma unroll
                for (int j = 0; j < W / 2; ++j) reinterpret_cast<float4 *>(m[u].ch)[j] = q[j];
            }
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
            if (u < n)
#pragma unroll
                for (int i = 0; i < W; ++i) c[i] = m[u].ch[i].x < 0.f ? m[u].ch[i].y : fmaf(m[u].ch[i].x, c[i], m[u].ch[i].y);
        k += n * step;
    }
}

// The state before every piece, where pieces are many: a CTA takes a channel unit, its 32
// warps a run of pieces each. They compose their maps, then the runs before their own, and
// walk their maps again.
template <int W>
__global__ void __launch_bounds__(1024) scan_carry_kernel(const void *maps, float *carry, int pieces, int units, int backward) {
    __shared__ Map<W> runs[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long pitch = (long long)units * 32, at = (long long)blockIdx.x * 32 + lane;
    const Map<W> *m = static_cast<const Map<W> *>(maps) + at;
    const int per = (pieces + 31) / 32, p0 = min(warp * per, pieces), p1 = min(p0 + per, pieces);
    auto place = [&](int j) { return (long long)(backward ? pieces - 1 - j : j) * pitch; };
    Map<W> run;
#pragma unroll
    for (int i = 0; i < W; ++i) run.ch[i] = make_float2(1.f, 0.f);
    for (int j = p0; j < p1; j += 4) {
        Map<W> q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (j + u < p1) q[u] = m[place(j + u)];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (j + u < p1)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float2 n = q[u].ch[i];
                    run.ch[i] = n.x < 0.f ? n : make_float2(run.ch[i].x < 0.f ? -1.f : run.ch[i].x * n.x, fmaf(n.x, run.ch[i].y, n.y));
                }
    }
    runs[warp][lane] = run;
    __syncthreads();
    float c[W];
    vset(c, 0.f);
    auto through = [&](const Map<W> &n) {
#pragma unroll
        for (int i = 0; i < W; ++i) c[i] = n.ch[i].x < 0.f ? n.ch[i].y : fmaf(n.ch[i].x, c[i], n.ch[i].y);
    };
    for (int w = 0; w < warp; ++w) through(runs[w][lane]);
    for (int j = p0; j < p1; j += 4) {
        Map<W> q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (j + u < p1) q[u] = m[place(j + u)];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (j + u < p1) {
#pragma unroll
                for (int i = 0; i < W; ++i) carry[(place(j + u) + at) * W + i] = c[i];
                through(q[u]);
            }
    }
}

template <int W>
__device__ __forceinline__ void enter_cut(const ScanCut &cut, int c0, int units, int first, int piece, int step, float (&c)[W]) {
    if (!cut.carry) {
        compose(lane_map<W>(cut, c0), (long long)units * 32, first, piece, step, c);
        return;
    }
    const float *p = cut.carry + ((long long)piece * units * 32 + c0 / W) * W;
#pragma unroll
    for (int i = 0; i < W; ++i) c[i] = p[i];
}
// The state before (backward: behind) a piece, from the carry kernel or composed here of the
// maps from piece `first` on. Without maps (a cut after the host's offsets, none of which the
// device's may share) zeros; lanes of 4 bytes never have any.
template <int LB, int W>
__device__ __forceinline__ void enter(const ScanCut &cut, int c0, int units, int first, int piece, int step, float (&c)[W]) {
    if constexpr (LB == 8) {
        if (cut.maps) {
            enter_cut(cut, c0, units, first, piece, step, c);
            return;
        }
    }
    vset(c, 0.f);
}
// ---------------------------------------------------------------- forward
// One step of a lane's channels: a, and what is added to a h.
template <typename T, bool SIG, typename R, int W>
__device__ __forceinline__ void step_fwd(const R &ring, int slot, int s, int r, float lb, float (&a)[W], float (&v)[W]) {
    float g[W], b[W];
    ring.get(slot, 0, s, r, v);
    ring.get(slot, 1, s, r, g);
    decays<T, SIG>(g, lb, a, b);
    if (SIG) vmul(v, b, v);
}

// The same of rows s0 .. s0+UN-1 of a stage, one operation of all of them after the other: a
// walker has its scheduler almost to itself, so neighbouring instructions have to be
// independent (31744 x 12288: 5 % of the call's time).
template <typename T, bool SIG, int UN, typename R, int W>
__device__ __forceinline__ void steps_fwd(const R &ring, int slot, int s0, int r, float lb, float (&a)[UN][W], float (&v)[UN][W]) {
    float b[UN][W];
#pragma unroll
    for (int s = 0; s < UN; ++s) ring.get(slot, 1, s0 + s, r + s, a[s]);
#pragma unroll
    for (int s = 0; s < UN; ++s) ring.get(slot, 0, s0 + s, r + s, v[s]);
    decays<T, SIG, UN>(a, lb, b);
    if (SIG)
#pragma unroll
        for (int s = 0; s < UN; ++s) vmul(v[s], b[s], v[s]);
}

template <typename T, int G, int LB, bool SIG>
__global__ void __launch_bounds__(32) scan_fwd_kernel(const __grid_constant__ ScanParams p) {
    using RN = ScanRing<T, G, LB, 2>;
    constexpr int W = RN::W, S = kStage, ST = ring_stages(LB, 2), UN = unrolled<G>(), TC = walk_channels<T, LB>();
    extern __shared__ __align__(16) char dyn[];
    const int lane = threadIdx.x, D = p.D, R = p.span.R, units = (D + TC - 1) / TC;
    const int piece = blockIdx.x / units, c0 = (blockIdx.x - piece * units) * TC, c = c0 + lane * W;
    int b, e;
    piece_rows(p.cut, p.span, piece, b, e);
    RN ring{dyn, {walk_tensor<T>(p.x, p.x_stride, c0, D, R), walk_tensor<T>(p.g, p.g_stride, c0, D, R)},
            min(TC, D - c0) * (int)sizeof(T), lane};
    ring.begin(0, b);
    ring.begin(1, b);
    auto load = [&](int slot, int row) {
        ring.template load<1>(slot, 0, row, b, e);
        ring.template load<1>(slot, 1, row, b, e);
    };
    if (b < e) {
#pragma unroll 1
        for (int k = 0; k < ST - 1; ++k) {
            if (b + k * S < e) load(k, b + k * S);
            cp_async_commit();
        }
    }
    hand_through<W>(p.span, piece, p.cut.pieces, lane, c, D, 1, p.sT, p.s0);
    if (b >= e) return;
    Seq q = seq_of(p.span, b, lane);
    float h[W];
    if (q.start < b) enter<LB>(p.cut, c, units, piece_of(p.cut, p.span, q.start), piece, 1, h);
    else get_state(p.s0, q.n, c, D, h);
    // behind the last row of a sequence
    auto close = [&](int row) {
        if (p.sT) put_state(p.sT, q.n, c, D, h);
        if (row < e) {
            q = seq_of(p.span, row, lane);
            get_state(p.s0, q.n, c, D, h);
        }
    };
    T *out = static_cast<T *>(p.h) + (long long)b * D;
    int slot = 0, next = ST - 1;
#pragma unroll 1
    for (int r = b; r < e; r += S) {
        cp_async_wait_group<ST - 2>();
        __syncwarp();
        const int ahead = r + (ST - 1) * S;
        if (ahead < e) load(next, ahead);
        cp_async_commit();
        auto one = [&](int s) {
            float a[W], v[W];
            step_fwd<T, SIG>(ring, slot, s, r + s, p.lb, a, v);
            vfma(a, h, v, h);
            put_row<G>(out + (long long)s * D, c, D, lane, h);
        };
        if (min(q.end, e) >= r + S) {
            auto rows = [&](int s0) {  // the decays of UN rows, then the rows
                float a[UN][W], v[UN][W];
                steps_fwd<T, SIG, UN>(ring, slot, s0, r + s0, p.lb, a, v);
#pragma unroll
                for (int s = 0; s < UN; ++s) vfma(a[s], s ? v[s - 1] : h, v[s], v[s]);
#pragma unroll
                for (int s = 0; s < UN; ++s) put_row<G>(out + (long long)(s0 + s) * D, c, D, lane, v[s]);
#pragma unroll
                for (int i = 0; i < W; ++i) h[i] = v[UN - 1][i];
            };
            if constexpr (UN == S) {
                rows(0);
            } else {
#pragma unroll 1
                for (int s0 = 0; s0 < S; s0 += UN) rows(s0);
            }
            if (q.end == r + S) close(r + S);
        } else {
            const int n = min(S, e - r);
#pragma unroll 1
            for (int s = 0; s < n; ++s) {
                one(s);
                if (q.end == r + s + 1) close(r + s + 1);
            }
        }
        out += (long long)S * D;
        next = slot;
        slot = slot + 1 == ST ? 0 : slot + 1;
    }
}

// The map of a piece whose last sequence goes on behind it, over that sequence's rows.
template <typename T, int G, int LB, bool SIG>
__global__ void __launch_bounds__(32) scan_reduce_kernel(const __grid_constant__ ScanParams p) {
    using RN = ScanRing<T, G, LB, 2>;
    constexpr int W = RN::W, S = kStage, ST = ring_stages(LB, 2), UN = unrolled<G>(), TC = walk_channels<T, LB>();
    extern __shared__ __align__(16) char dyn[];
    const int lane = threadIdx.x, D = p.D, R = p.span.R, units = (D + TC - 1) / TC;
    const int piece = blockIdx.x / units, c0 = (blockIdx.x - piece * units) * TC, c = c0 + lane * W;
    int b, e;
    piece_rows(p.cut, p.span, piece, b, e);
    if (b >= e) return;
    const Seq q = seq_of(p.span, e - 1, lane);
    if (q.end <= e) return;
    const bool begins = q.start >= b;
    b = max(b, q.start);
    RN ring{dyn, {walk_tensor<T>(p.x, p.x_stride, c0, D, R), walk_tensor<T>(p.g, p.g_stride, c0, D, R)},
            min(TC, D - c0) * (int)sizeof(T), lane};
    ring.begin(0, b);
    ring.begin(1, b);
    auto load = [&](int slot, int row) {
        ring.template load<1>(slot, 0, row, b, e);
        ring.template load<1>(slot, 1, row, b, e);
    };
#pragma unroll 1
    for (int k = 0; k < ST - 1; ++k) {
        if (b + k * S < e) load(k, b + k * S);
        cp_async_commit();
    }
    float A[W], h[W];
    vset(A, 1.f);
    vset(h, 0.f);
    if (begins) get_state(p.s0, q.n, c, D, h);
    int slot = 0, next = ST - 1;
#pragma unroll 1
    for (int r = b; r < e; r += S) {
        cp_async_wait_group<ST - 2>();
        __syncwarp();
        const int ahead = r + (ST - 1) * S;
        if (ahead < e) load(next, ahead);
        cp_async_commit();
        auto one = [&](int s) {
            float a[W], v[W];
            step_fwd<T, SIG>(ring, slot, s, r + s, p.lb, a, v);
            vfma(a, h, v, h);
            vmul(A, a, A);
        };
        if (e >= r + S) {
            auto rows = [&](int s0) {
                float a[UN][W], v[UN][W];
#pragma unroll
                for (int s = 0; s < UN; ++s) step_fwd<T, SIG>(ring, slot, s0 + s, r + s0 + s, p.lb, a[s], v[s]);
#pragma unroll
                for (int s = 0; s < UN; ++s) {
                    vfma(a[s], h, v[s], h);
                    vmul(A, a[s], A);
                }
            };
            if constexpr (UN == S) {
                rows(0);
            } else {
#pragma unroll 1
                for (int s0 = 0; s0 < S; s0 += UN) rows(s0);
            }
        } else {
#pragma unroll 1
            for (int s = 0; s < e - r; ++s) one(s);
        }
        next = slot;
        slot = slot + 1 == ST ? 0 : slot + 1;
    }
    Map<W> m;
#pragma unroll
    for (int i = 0; i < W; ++i) m.ch[i] = make_float2(begins ? -1.f : A[i], h[i]);
    lane_map<W>(p.cut, c)[(long long)piece * units * 32] = m;
}

// ---------------------------------------------------------------- backward
// With k the cotangent that row t+1 hands back (behind a sequence's last row dfinal):
//     d = dout_t + k,  dx = d (or (1 - a) d),  dg = d a h_{t-1} (0 below the bound), or
//     d (h_{t-1} - x) a (1 - a),  k <- a d,  and dinitial is what the first row hands back.
// The same walk from the last row to the first; h is the forward's output, so h_{t-1}
// carries the rounding of its type (half a step, as the gradient itself does), which saves
// the forward's recomputation and the reading of x in the log form.
template <typename T, int G, int LB, bool SIG>
__global__ void __launch_bounds__(32) scan_bwd_kernel(const __grid_constant__ ScanBwdParams p) {
    constexpr int N = SIG ? 4 : 3;
    using RN = ScanRing<T, G, LB, N>;
    constexpr int W = RN::W, S = kStage, ST = ring_stages(LB, N), UN = unrolled<G>(), TC = walk_channels<T, LB>();
    extern __shared__ __align__(16) char dyn[];
    const int lane = threadIdx.x, D = p.D, R = p.span.R, units = (D + TC - 1) / TC;
    const int place = blockIdx.x / units, piece = p.cut.pieces - 1 - place, c0 = (blockIdx.x - place * units) * TC, c = c0 + lane * W;
    int b, e;
    piece_rows(p.cut, p.span, piece, b, e);
    RN ring{dyn, {walk_tensor<T>(p.g, p.g_stride, c0, D, R), walk_tensor<T>(p.dout, p.dout_stride, c0, D, R),
                  walk_tensor<T>(p.h, p.h_stride, c0, D, R)}, min(TC, D - c0) * (int)sizeof(T), lane};
    if (SIG) ring.t[N - 1] = walk_tensor<T>(p.x, p.x_stride, c0, D, R);
    ring.begin(0, e - S);
    ring.begin(1, e - S);
    ring.begin(2, e - S - 1);
    if (SIG) ring.begin(N - 1, e - S);
    // a stage's rows from `row` on, of h the rows before them
    auto load = [&](int slot, int row) {
        ring.template load<-1>(slot, 0, row, b, e);
        ring.template load<-1>(slot, 1, row, b, e);
        ring.template load<-1>(slot, 2, row - 1, max(b - 1, 0), e - 1);
        if (SIG) ring.template load<-1>(slot, N - 1, row, b, e);
    };
    if (b < e) {
#pragma unroll 1
        for (int k = 0; k < ST - 1; ++k) {
            if (e - k * S > b) load(k, e - (k + 1) * S);
            cp_async_commit();
        }
    }
    hand_through<W>(p.span, piece, p.cut.pieces, lane, c, D, 1, p.ds0, p.dsT);
    if (b >= e) return;
    Seq q = seq_of(p.span, e - 1, lane);
    float k[W];
    if (q.end > e) enter<LB>(p.cut, c, units, piece_of(p.cut, p.span, q.end - 1), piece, -1, k);
    else get_state(p.dsT, q.n, c, D, k);
    int slot = 0, next = ST - 1;
#pragma unroll 1
    for (int r = e - S; r > b - S; r -= S) {
        cp_async_wait_group<ST - 2>();
        __syncwarp();
        const int ahead = r - (ST - 1) * S;
        if (ahead > b - S) load(next, ahead);
        cp_async_commit();
        auto one = [&](int s, bool first) {
            const int row = r + s;
            float g[W], d[W], hp[W], x[W], a[W], w[W], dg[W];
            ring.get(slot, 0, s, row, g);
            ring.get(slot, 1, s, row, d);
            if (first) get_state(p.s0, q.n, c, D, hp);
            else ring.get(slot, 2, s, row - 1, hp);
            if (SIG) ring.get(slot, N - 1, s, row, x);
            decays<T, SIG>(g, p.lb, a, w);
            vadd(d, k, d);
            vmul(a, d, k);
            if (SIG) {
#pragma unroll
                for (int i = 0; i < W; ++i) hp[i] -= x[i];
                vmul(w, d, d);
                vmul(w, k, dg);
                vmul(dg, hp, dg);
            } else {
                vmul(k, hp, dg);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (g[i] < p.lb) dg[i] = 0.f;
            }
            put_row<G>(static_cast<T *>(p.dx) + (long long)row * D, c, D, lane, d);
            put_row<G>(static_cast<T *>(p.dg) + (long long)row * D, c, D, lane, dg);
        };
        if (r >= b && q.start < r) {
#pragma unroll(UN)
            for (int s = S - 1; s >= 0; --s) one(s, false);
        } else {
#pragma unroll 1
            for (int s = S - 1; s >= 0 && r + s >= b; --s) {
                const bool first = r + s == q.start;
                one(s, first);
                if (first) {
                    if (p.ds0) put_state(p.ds0, q.n, c, D, k);
                    if (r + s > b) {
                        q = seq_of(p.span, r + s - 1, lane);
                        get_state(p.dsT, q.n, c, D, k);
                    }
                }
            }
        }
        next = slot;
        slot = slot + 1 == ST ? 0 : slot + 1;
    }
}

// The map, run backwards, of a piece whose first sequence began before it.
template <typename T, int G, int LB, bool SIG>
__global__ void __launch_bounds__(32) scan_reduce_bwd_kernel(const __grid_constant__ ScanBwdParams p) {
    using RN = ScanRing<T, G, LB, 2>;
    constexpr int W = RN::W, S = kStage, ST = ring_stages(LB, 2), UN = unrolled<G>(), TC = walk_channels<T, LB>();
    extern __shared__ __align__(16) char dyn[];
    const int lane = threadIdx.x, D = p.D, R = p.span.R, units = (D + TC - 1) / TC;
    const int piece = blockIdx.x / units, c0 = (blockIdx.x - piece * units) * TC, c = c0 + lane * W;
    int b, e;
    piece_rows(p.cut, p.span, piece, b, e);
    if (b >= e) return;
    const Seq q = seq_of(p.span, b, lane);
    if (q.start >= b) return;
    const bool ends = q.end <= e;
    e = min(e, q.end);
    RN ring{dyn, {walk_tensor<T>(p.g, p.g_stride, c0, D, R), walk_tensor<T>(p.dout, p.dout_stride, c0, D, R)},
            min(TC, D - c0) * (int)sizeof(T), lane};
    ring.begin(0, e - S);
    ring.begin(1, e - S);
    auto load = [&](int slot, int row) {
        ring.template load<-1>(slot, 0, row, b, e);
        ring.template load<-1>(slot, 1, row, b, e);
    };
#pragma unroll 1
    for (int k = 0; k < ST - 1; ++k) {
        if (e - k * S > b) load(k, e - (k + 1) * S);
        cp_async_commit();
    }
    float A[W], h[W];
    vset(A, 1.f);
    vset(h, 0.f);
    if (ends) get_state(p.dsT, q.n, c, D, h);
    int slot = 0, next = ST - 1;
#pragma unroll 1
    for (int r = e - S; r > b - S; r -= S) {
        cp_async_wait_group<ST - 2>();
        __syncwarp();
        const int ahead = r - (ST - 1) * S;
        if (ahead > b - S) load(next, ahead);
        cp_async_commit();
        auto one = [&](int s) {
            float g[W], d[W], a[W], w[W];
            ring.get(slot, 0, s, r + s, g);
            ring.get(slot, 1, s, r + s, d);
            decays<T, SIG>(g, p.lb, a, w);
            vadd(d, h, d);
            vmul(a, d, h);
            vmul(A, a, A);
        };
        if (r >= b) {
#pragma unroll(UN)
            for (int s = S - 1; s >= 0; --s) one(s);
        } else {
#pragma unroll 1
            for (int s = S - 1; r + s >= b; --s) one(s);
        }
        next = slot;
        slot = slot + 1 == ST ? 0 : slot + 1;
    }
    Map<W> m;
#pragma unroll
    for (int i = 0; i < W; ++i) m.ch[i] = make_float2(ends ? -1.f : A[i], h[i]);
    lane_map<W>(p.cut, c)[(long long)piece * units * 32] = m;
}

// ---------------------------------------------------------------- single token
// 16 bytes of state a thread where everything is aligned, one channel otherwise.
template <typename T, bool AL, bool SIG>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ ScanStepParams p) {
    constexpr int W = AL ? 4 : 1;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int per = p.D / W, n = (int)(i / per), c = (int)(i - (long long)n * per) * W;
    if (n >= p.N) return;
    const T *xp = static_cast<const T *>(p.x) + n * p.x_stride + c, *gp = static_cast<const T *>(p.g) + n * p.g_stride + c;
    const long long at = (long long)n * p.D + c;
    T x[W], g[W], o[W];
    float h[W];
    if constexpr (AL) {
        *reinterpret_cast<float4 *>(h) = *reinterpret_cast<const float4 *>(p.state + at);
        using V = typename std::conditional<sizeof(T) == 2, uint2, uint4>::type;
        *reinterpret_cast<V *>(x) = *reinterpret_cast<const V *>(xp);
        *reinterpret_cast<V *>(g) = *reinterpret_cast<const V *>(gp);
    } else {
        h[0] = p.state[at]; x[0] = xp[0]; g[0] = gp[0];
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float a, b;
        decay<T, SIG>(to_f32(g[j]), p.lb, a, b);
        h[j] = fmaf(a, h[j], SIG ? b * to_f32(x[j]) : to_f32(x[j]));
        o[j] = from_f32<T>(h[j]);
    }
    if constexpr (AL) {
        using V = typename std::conditional<sizeof(T) == 2, uint2, uint4>::type;
        *reinterpret_cast<float4 *>(p.state_out + at) = *reinterpret_cast<const float4 *>(h);
        *reinterpret_cast<V *>(static_cast<T *>(p.h) + at) = *reinterpret_cast<const V *>(o);
    } else {
        p.state_out[at] = h[0];
        static_cast<T *>(p.h)[at] = o[0];
    }
}

// ---------------------------------------------------------------- host
int units_of(int D, bool bf16, int lb) {
    const int tc = bf16 ? 16 * lb : 8 * lb;
    return (D + tc - 1) / tc;
}

// Pieces of `each` rows; rows + each may pass 32 bits.
int pieces_of(int rows, int each) { return (int)(((long long)rows + each - 1) / each); }

// How the rows are cut for walkers of `lb` bytes a lane. Whole sequences where walkers of
// whole sequences come to half of those that can run at a time, none more than three times
// as long as the average (one pass; without the lengths on the host a packed batch is taken
// to be ragged); otherwise pieces of equal length, for one full wave of walkers and of
// kMinPiece rows at least. Forward and backward (log form) of 2048 channels in bf16, where 64 pieces are
// a wave, us, whole against cut:
//   32 x 1024 rows 62, 106 against 78, 134;  31 x 1024 60, 105 against 76, 127 (cut, the far side of
//   the rule);  16 x 1024 58, 102 against 51, 76: the two sides meet between a quarter and half
//   32 packed of 1000 rows on average, longest 1000: 62, 106 against 97, 155;  2000: 114, 199
//   against 101, 152 (whole);  3000: 168, 296 against 100, 152
//   64 packed, longest 2000: 157, 273 against 188, 284;  3000: 204, 363 against 192, 287
//   512 packed of 128 rows 125, 211 against 146, 248 (cut: more than four waves)
ScanCut cut_for(const RowSpan &sp, const int32_t *cu_host, int D, bool bf16, int lb) {
    const int units = units_of(D, bf16, lb);
    const long long want = kWalkerSlots > units ? kWalkerSlots / units : 1;  // pieces of a full wave
    ScanCut c{};
    c.lb = lb;
    if (sp.R == 0) {
        c.kind = kCutRows; c.pieces = 1; c.rows = 1;
        return c;
    }
    auto stages = [](long long rows) { return (int)((rows + kStage - 1) / kStage * kStage); };
    if (!sp.cu) {
        if (2LL * sp.N >= want || sp.T <= 2 * kMinPiece) {
            // whole sequences, several to a walker where there are many
            const long long each = (sp.N + want - 1) / want;
            c.kind = kCutRows;
            c.rows = (int)(each * sp.T);
            c.pieces = (int)((sp.N + each - 1) / each);
            return c;
        }
        const int per = (int)(want / sp.N);
        c.kind = kCutBatch;
        c.rows = stages(sp.T / per > kMinPiece ? (sp.T + per - 1) / per : kMinPiece);
        c.per = pieces_of(sp.T, c.rows);
        c.pieces = sp.N * c.per;
        c.carries = c.per > 1;
        return c;
    }
    if (cu_host && 2LL * sp.N >= want && sp.N <= 4 * want) {
        int longest = 0;
        for (int n = 0; n < sp.N; ++n) longest = longest < cu_host[n + 1] - cu_host[n] ? cu_host[n + 1] - cu_host[n] : longest;
        if ((long long)longest * sp.N <= 3LL * sp.R || longest <= 2 * kMinPiece) {
            c.kind = kCutSeqs; c.pieces = sp.N;
            return c;
        }
    }
    c.kind = kCutRows;
    c.rows = stages(sp.R / want > kMinPiece ? (sp.R + want - 1) / want : kMinPiece);
    c.pieces = pieces_of(sp.R, c.rows);
    c.carries = c.pieces > 1;
    return c;
}

// A walker composes up to this many maps itself; beyond, a kernel between the two passes
// hands every walker its state. Forward of bf16, us, without it and with it: 129 pieces 64 and
// 67, 207 and 259 the same, 345 pieces 109 and 105, 518 pieces 104 and 87, 1036 pieces 106 and 65.
constexpr int kOwnMaps = 256;

// Scratch: the maps, then the states before the pieces.
size_t map_bytes(const ScanCut &c, int D, bool bf16) { return sizeof(float2) * (size_t)c.pieces * units_of(D, bf16, c.lb) * (bf16 ? 16 : 8) * c.lb; }

void lay_out(ScanCut *c, int D, bool bf16, void *workspace) {
    c->maps = c->carries ? workspace : nullptr;
    c->carry = c->carries && c->pieces > kOwnMaps ? reinterpret_cast<float *>(static_cast<char *>(workspace) + map_bytes(*c, D, bf16)) : nullptr;
}

// Lanes of 8 bytes take about two thirds of the instructions an element; lanes of 4 make
// twice the walkers, and are taken where they save the cut along time (31744 x 12288 packed
// of four sequences: 511 us in one pass, 637 with lanes of 8 in two; x 12292, by 8 bytes: 859
// against 996), but for accesses of less than 8 bytes (x 12289: 2017 against 1021). At the least
// number of walkers that take them, 16 x 1024 x 2048, the forward gains (41 against 51) and the
// backward loses (88 against 76).
ScanCut scan_cut(const RowSpan &sp, const int32_t *cu_host, int D, bool bf16, int g) {
    const ScanCut wide = cut_for(sp, cu_host, D, bf16, 8);
    if (!wide.carries || g < 8) return wide;
    const ScanCut narrow = cut_for(sp, cu_host, D, bf16, 4);
    return narrow.carries ? wide : narrow;
}

template <int W> cudaError_t run_carry(const ScanCut &c, int D, bool bf16, int backward, cudaStream_t st) {
    if (!c.carry) return cudaSuccess;
    const int units = units_of(D, bf16, c.lb);
    count_launch();
    scan_carry_kernel<W><<<units, 1024, 0, st>>>(c.maps, c.carry, c.pieces, units, backward);
    return cudaGetLastError();
}

// Lanes of 4 bytes come with one pass over the rows and wide accesses (see scan_cut).
template <typename T, int G, int LB, bool SIG> cudaError_t run_fwd_lb(const ScanParams &p, cudaStream_t st) {
    constexpr int ring = ScanRing<T, G, LB, 2>::BYTES;
    const int units = units_of(p.D, sizeof(T) == 2, LB);
    cudaError_t e = cudaSuccess;
    if constexpr (LB == 8) {
        if (p.cut.carries) e = run_walk(scan_reduce_kernel<T, G, LB, SIG>, p, p.cut.pieces, units, ring, st);
        if (e == cudaSuccess) e = run_carry<lane_channels<T, LB>()>(p.cut, p.D, sizeof(T) == 2, 0, st);
    }
    return e != cudaSuccess ? e : run_walk(scan_fwd_kernel<T, G, LB, SIG>, p, p.cut.pieces, units, ring, st);
}
template <typename T, int G, int LB, bool SIG> cudaError_t run_bwd_lb(const ScanBwdParams &p, cudaStream_t st) {
    const int units = units_of(p.D, sizeof(T) == 2, LB);
    cudaError_t e = cudaSuccess;
    if constexpr (LB == 8) {
        if (p.cut.carries) e = run_walk(scan_reduce_bwd_kernel<T, G, LB, SIG>, p, p.cut.pieces, units, ScanRing<T, G, LB, 2>::BYTES, st);
        if (e == cudaSuccess) e = run_carry<lane_channels<T, LB>()>(p.cut, p.D, sizeof(T) == 2, 1, st);
    }
    return e != cudaSuccess ? e : run_walk(scan_bwd_kernel<T, G, LB, SIG>, p, p.cut.pieces, units, ScanRing<T, G, LB, SIG ? 4 : 3>::BYTES, st);
}
template <typename T, int G, bool SIG> cudaError_t run_fwd(const ScanParams &p, cudaStream_t st) {
    if constexpr (G >= 8)
        if (p.cut.lb == 4) return run_fwd_lb<T, G, 4, SIG>(p, st);
    return run_fwd_lb<T, G, 8, SIG>(p, st);
}
template <typename T, int G, bool SIG> cudaError_t run_bwd(const ScanBwdParams &p, cudaStream_t st) {
    if constexpr (G >= 8)
        if (p.cut.lb == 4) return run_bwd_lb<T, G, 4, SIG>(p, st);
    return run_bwd_lb<T, G, 8, SIG>(p, st);
}
template <typename T, bool AL, bool SIG> cudaError_t run_step(const ScanStepParams &p, cudaStream_t st) {
    const long long threads = (long long)p.N * (p.D / (AL ? 4 : 1));
    count_launch();
    scan_step_kernel<T, AL, SIG><<<(unsigned)((threads + 127) / 128), 128, 0, st>>>(p);
    return cudaGetLastError();
}

// Runs F<T, G, SIG> for the types and layouts of a call.
#define KDA_SCAN_SIG(F, T, G, sig) return sig ? F<T, G, true>(p, st) : F<T, G, false>(p, st);
#define KDA_SCAN_PICK(F, p, bf16, g, sig, st)                    \
    if (bf16) {                                                  \
        if (g == 16) KDA_SCAN_SIG(F, __nv_bfloat16, 16, sig)     \
        if (g == 8) KDA_SCAN_SIG(F, __nv_bfloat16, 8, sig)       \
        if (g == 4) KDA_SCAN_SIG(F, __nv_bfloat16, 4, sig)       \
        KDA_SCAN_SIG(F, __nv_bfloat16, 2, sig)                   \
    }                                                            \
    if (g == 16) KDA_SCAN_SIG(F, float, 16, sig)                 \
    if (g == 8) KDA_SCAN_SIG(F, float, 8, sig)                   \
    KDA_SCAN_SIG(F, float, 4, sig)

}  // namespace

size_t scan_workspace_bytes(const RowSpan &span, const int32_t *cu_host, int D, bool bf16) {
    // of the wider walkers: whether the narrower are taken goes by alignment too
    const ScanCut c = cut_for(span, cu_host, D, bf16, 8);
    if (!c.carries) return 0;
    const size_t maps = map_bytes(c, D, bf16);
    return c.pieces > kOwnMaps ? maps + maps / 2 : maps;
}

cudaError_t launch_scan(ScanParams p, const int32_t *cu_host, bool bf16, bool sigmoid, void *workspace, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4;
    RowAccess ac;
    ac.rows(p.x, p.x_stride, p.D, esz);
    ac.rows(p.g, p.g_stride, p.D, esz);
    ac.rows(p.h, p.D, p.D, esz);
    p.cut = scan_cut(p.span, cu_host, p.D, bf16, ac.g());
    lay_out(&p.cut, p.D, bf16, workspace);
    KDA_SCAN_PICK(run_fwd, p, bf16, ac.g(), sigmoid, st)
}

cudaError_t launch_scan_bwd(ScanBwdParams p, const int32_t *cu_host, bool bf16, bool sigmoid, void *workspace, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4;
    RowAccess ac;
    if (sigmoid) ac.rows(p.x, p.x_stride, p.D, esz);
    ac.rows(p.g, p.g_stride, p.D, esz);
    ac.rows(p.h, p.h_stride, p.D, esz);
    ac.rows(p.dout, p.dout_stride, p.D, esz);
    ac.rows(p.dx, p.D, p.D, esz);
    ac.rows(p.dg, p.D, p.D, esz);
    p.cut = scan_cut(p.span, cu_host, p.D, bf16, ac.g());
    lay_out(&p.cut, p.D, bf16, workspace);
    KDA_SCAN_PICK(run_bwd, p, bf16, ac.g(), sigmoid, st)
}

cudaError_t launch_scan_step(const ScanStepParams &p, bool bf16, bool sigmoid, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4;
    RowAccess ac;
    ac.rows(p.x, p.x_stride, p.D, esz);
    ac.rows(p.g, p.g_stride, p.D, esz);
    ac.rows(p.h, p.D, p.D, esz);
    ac.rows(p.state, p.D, p.D, 4);
    ac.rows(p.state_out, p.D, p.D, 4);
    if (bf16) {
        if (ac.g() == 16) return sigmoid ? run_step<__nv_bfloat16, true, true>(p, st) : run_step<__nv_bfloat16, true, false>(p, st);
        return sigmoid ? run_step<__nv_bfloat16, false, true>(p, st) : run_step<__nv_bfloat16, false, false>(p, st);
    }
    if (ac.g() == 16) return sigmoid ? run_step<float, true, true>(p, st) : run_step<float, true, false>(p, st);
    return sigmoid ? run_step<float, false, true>(p, st) : run_step<float, false, false>(p, st);
}

}  // namespace kda

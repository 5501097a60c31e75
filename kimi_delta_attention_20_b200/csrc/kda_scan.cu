// Gated linear recurrence over packed sequences, per channel:
//     log form      a = exp(max(g, lb)),  h_t = a_t h_{t-1} + x_t
//     sigmoid form  a = sigmoid(g),       h_t = a_t h_{t-1} + (1 - a_t) x_t
// its backward pass and its single token.
//
// A run of steps is the map c -> A c + H of the state before it (A the product of its a,
// H its result from zero), and maps compose, so time can be cut: the rows of all
// sequences form one axis that is cut into chunks of L rows whatever the sequences'
// lengths; a sequence's first row drops what came before (its map has A = 0, and the
// initial state enters H). A CTA takes a chunk of 128 channels: each warp a few
// consecutive rows, four channels a lane, everything in registers. Once its rows are
// loaded the CTA
//   1. forms the map of each warp's rows and, from these, of the chunk, and publishes it;
//   2. gets the state before the chunk: chunks form groups; it composes the maps of the
//      chunks of its group before it onto the state behind the previous group, which the
//      last chunk of that group published;
//   3. walks its rows again from the state before each warp, as the definition says.
// So x and g are read once and h is written once (6 bytes an element in bf16), which is
// the floor. What is composed, and in which order, goes by positions alone: results do
// not depend on timing. Chunks are handed out by a ticket in the order of the chain, so a
// CTA only waits for CTAs that are already running; every wait has a limit.
#include "kda_layer.cuh"
#include "kda_sm100.cuh"

namespace kda {

namespace {

constexpr int kScanWarps = 8, kScanThreads = 32 * kScanWarps;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ unsigned ld_acquire(const unsigned *p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(unsigned *p, unsigned v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Waits until *flag is set. Gives up after 2 s, or once another wait has given up.
__device__ __forceinline__ void wait_flag(const unsigned *flag, int *status) {
    if (ld_acquire(flag)) return;
    const uint64_t t0 = sm100::globaltimer_ns();
    while (!ld_acquire(flag)) {
        if (sm100::globaltimer_ns() - t0 > kWaitLimitNs || *reinterpret_cast<volatile int *>(status)) {
            *reinterpret_cast<volatile int *>(status) = 1;
            return;
        }
        __nanosleep(64);
    }
}

// a of the gate input, and the weight of x in the sigmoid form: 1 - a without the
// cancellation, since a is close to 1 where memories are long.
template <bool SIG> __device__ __forceinline__ void decay(float g, int has_lb, float lb, float &a, float &b) {
    if (SIG) {
        const float e = expf(-fabsf(g)), r = 1.f / (1.f + e);
        a = g >= 0.f ? r : e * r;
        b = g >= 0.f ? e * r : r;
        if (!(g == g)) a = b = g;
    } else {
        a = expf(has_lb && g < lb ? lb : g);
        b = 1.f;
    }
}

// Shared memory of a CTA: the maps of its warps and of the window that it composes.
template <int L> struct ScanShared {
    RowMap<L> map;
    float4 A[kScanWarps][32], H[kScanWarps][32];
    float4 wA[kScanWarps][32], wH[kScanWarps][32], init[32];
    int reset[kScanWarps];
    unsigned ticket;
};

__device__ __forceinline__ void put4(float4 &d, const float (&v)[4]) { d = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void get4(const float4 &s, float (&v)[4]) { v[0] = s.x; v[1] = s.y; v[2] = s.z; v[3] = s.w; }

// The chunk and channel tile of this CTA.
template <int L> __device__ __forceinline__ void take_item(ScanShared<L> &sm, const ScanChain &ch, int &chunk, int &tile) {
    unsigned item = blockIdx.x;
    if (ch.chunks > 1) {
        if (threadIdx.x == 0) sm.ticket = atomicAdd(ch.ticket, 1u);
        __syncthreads();
        item = sm.ticket;
    }
    chunk = (int)(item / (unsigned)ch.tiles);
    tile = (int)(item - (unsigned)chunk * (unsigned)ch.tiles);
}

// Joins the maps of the CTA's warps (warp order is chain order), publishes the chunk's,
// and returns the state before this warp's rows. A, H: this warp's map, `reset` whether a
// sequence begins in it (what comes before then has no part, not even as 0 x inf).
// carry: whether the chunk continues a sequence, which began in chunk `from`.
template <int L>
__device__ __forceinline__ void join(ScanShared<L> &sm, const ScanChain &ch, int chunk, int tile, bool carry, int from,
                                     const float (&A)[4], const float (&H)[4], bool reset, float (&c)[4]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    put4(sm.A[warp][lane], A);
    put4(sm.H[warp][lane], H);
    if (lane == 0) sm.reset[warp] = reset;
    __syncthreads();
    float PA[4] = {1.f, 1.f, 1.f, 1.f}, PH[4] = {0.f, 0.f, 0.f, 0.f};
    bool cut = false;  // a sequence begins before this warp's rows
    for (int w = 0; w < warp; ++w) {
        float a[4], h[4];
        get4(sm.A[w][lane], a);
        get4(sm.H[w][lane], h);
        if (sm.reset[w]) {
            cut = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) { PA[i] = 0.f; PH[i] = h[i]; }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) { PH[i] = fmaf(a[i], PH[i], h[i]); PA[i] *= a[i]; }
        }
    }
    const int group = chunk / ch.group, at = chunk - group * ch.group;
    if (warp == kScanWarps - 1 && at != ch.group - 1 && chunk + 1 < ch.chunks) {
        float2 *agg = ch.agg + ((long long)chunk * ch.tiles + tile) * kTileChannels + lane * 4;
        float tA[4], tH[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            tA[i] = reset ? 0.f : PA[i] * A[i];
            tH[i] = reset ? H[i] : fmaf(A[i], PH[i], H[i]);
        }
        __stcg(reinterpret_cast<float4 *>(agg), make_float4(tA[0], tH[0], tA[1], tH[1]));
        __stcg(reinterpret_cast<float4 *>(agg) + 1, make_float4(tA[2], tH[2], tA[3], tH[3]));
        __threadfence();
        __syncwarp();
        if (lane == 0 && !(ch.stall && chunk == 0)) st_release(ch.flags + (long long)chunk * ch.tiles + tile, 1u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = 0.f;
    if (carry) {
        // the window: from the chunk where the sequence began or from the group's first
        const int g0 = group * ch.group;
        const bool whole = from < g0;  // the sequence reaches back beyond the group
        const int first = whole ? g0 : min(from, chunk), n = chunk - first;
        const int per = (n + kScanWarps - 1) / kScanWarps;
        const int b = min(warp * per, n), e = min(b + per, n);
        if (b + lane < e) wait_flag(ch.flags + (long long)(first + b + lane) * ch.tiles + tile, ch.status);
        if (warp == kScanWarps - 1 && whole) {
            if (lane == 0) wait_flag(ch.flags + (long long)(g0 - 1) * ch.tiles + tile, ch.status);
            __syncwarp();
            const float *inc = ch.inc + ((long long)(group - 1) * ch.tiles + tile) * kTileChannels;
            sm.init[lane] = __ldcg(reinterpret_cast<const float4 *>(inc) + lane);
        }
        __syncwarp();
        float wA[4] = {1.f, 1.f, 1.f, 1.f}, wH[4] = {0.f, 0.f, 0.f, 0.f};
        const float4 *agg = reinterpret_cast<const float4 *>(ch.agg + ((long long)(first + b) * ch.tiles + tile) * kTileChannels) + lane * 2;
#pragma unroll 4
        for (int k = b; k < e; ++k, agg += (long long)ch.tiles * (kTileChannels / 2)) {
            const float4 p = __ldcg(agg), q = __ldcg(agg + 1);
            wH[0] = fmaf(p.x, wH[0], p.y); wA[0] *= p.x;
            wH[1] = fmaf(p.z, wH[1], p.w); wA[1] *= p.z;
            wH[2] = fmaf(q.x, wH[2], q.y); wA[2] *= q.x;
            wH[3] = fmaf(q.z, wH[3], q.w); wA[3] *= q.z;
        }
        put4(sm.wA[warp][lane], wA);
        put4(sm.wH[warp][lane], wH);
        __syncthreads();
        if (whole) get4(sm.init[lane], c);
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) {
            float a[4], h[4];
            get4(sm.wA[w][lane], a);
            get4(sm.wH[w][lane], h);
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = fmaf(a[i], c[i], h[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = cut ? PH[i] : fmaf(PA[i], c[i], PH[i]);
}

// The last chunk of a group publishes the state behind it (c: behind the last warp's rows).
__device__ __forceinline__ void publish_group(const ScanChain &ch, int chunk, int tile, const float (&c)[4]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = chunk / ch.group;
    if (warp != kScanWarps - 1 || chunk - group * ch.group != ch.group - 1 || chunk + 1 >= ch.chunks) return;
    float *inc = ch.inc + ((long long)group * ch.tiles + tile) * kTileChannels;
    __stcg(reinterpret_cast<float4 *>(inc) + lane, make_float4(c[0], c[1], c[2], c[3]));
    __threadfence();
    __syncwarp();
    if (lane == 0 && !(ch.stall && chunk == 0)) st_release(ch.flags + (long long)chunk * ch.tiles + tile, 1u);
}

// Bit s: a sequence starts (ends) at row s of the S rows.
template <int S> __device__ __forceinline__ unsigned row_bits(const int *rows, int lane) {
    return __ballot_sync(0xffffffffu, lane < S && rows[lane < S ? lane : 0] >= 0);
}

template <bool VEC>
__device__ __forceinline__ void store_state(float *rows, int n, int tile, int lane, int D, const float (&v)[4]) {
    store_row<float, VEC>(rows + (long long)n * D, tile, lane, D, v);
}

template <bool VEC>
__device__ __forceinline__ void state_or_zero(const float *rows, int n, int tile, int lane, int D, float (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = 0.f;
    if (rows) load_f32<VEC>(rows + (long long)n * D, tile, lane, D, v);
}

// ---------------------------------------------------------------- forward
template <typename T, bool VEC, bool SIG, int S>
__global__ void __launch_bounds__(kScanThreads, 2) scan_fwd_kernel(const __grid_constant__ ScanParams p) {
    constexpr int L = kScanWarps * S;
    __shared__ ScanShared<L> sm;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int chunk, tile;
    take_item(sm, p.chain, chunk, tile);
    const int row0 = chunk * L, wrow = row0 + warp * S, R = p.span.R, D = p.D;

    Raw4<T> xr[S], gr[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const bool ok = wrow + s < R;
        xr[s] = load_row<T, VEC>(static_cast<const T *>(p.x) + (long long)(wrow + s) * p.x_stride, tile, lane, D, ok);
        gr[s] = load_row<T, VEC>(static_cast<const T *>(p.g) + (long long)(wrow + s) * p.g_stride, tile, lane, D, ok);
    }
    // an empty sequence hands its state through
    fill_rows<L>(sm.map, p.span, row0, [&](int n) {
        if (!p.sT) return;
        const int c1 = min(D, (tile + 1) * kTileChannels);
        for (int c = tile * kTileChannels; c < c1; ++c) p.sT[(long long)n * D + c] = p.s0 ? p.s0[(long long)n * D + c] : 0.f;
    });
    if (R == 0) return;
    const unsigned starts = row_bits<S>(sm.map.start + warp * S, lane), ends = row_bits<S>(sm.map.end + warp * S, lane);

    float a[S][4], v[S][4], A[4] = {1.f, 1.f, 1.f, 1.f}, H[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float b;
            decay<SIG>(raw_get(gr[s], i), p.has_lb, p.lb, a[s][i], b);
            v[s][i] = SIG ? b * raw_get(xr[s], i) : raw_get(xr[s], i);
        }
        if (starts >> s & 1) {
            float h0[4];
            state_or_zero<VEC>(p.s0, sm.map.start[warp * S + s], tile, lane, D, h0);
#pragma unroll
            for (int i = 0; i < 4; ++i) { H[i] = fmaf(a[s][i], h0[i], v[s][i]); A[i] = 0.f; }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) { H[i] = fmaf(a[s][i], H[i], v[s][i]); A[i] *= a[s][i]; }
        }
    }
    float h[4];
    const bool carry = sm.map.first < row0;
    join<L>(sm, p.chain, chunk, tile, carry, max(sm.map.first, 0) / L, A, H, starts != 0, h);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (wrow + s < R) {
            if (starts >> s & 1) state_or_zero<VEC>(p.s0, sm.map.start[warp * S + s], tile, lane, D, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = fmaf(a[s][i], h[i], v[s][i]);
            store_row<T, VEC>(static_cast<T *>(p.h) + (long long)(wrow + s) * D, tile, lane, D, h);
            if (p.sT && (ends >> s & 1)) store_state<VEC>(p.sT, sm.map.end[warp * S + s], tile, lane, D, h);
        }
    }
    publish_group(p.chain, chunk, tile, h);
}

// ---------------------------------------------------------------- backward
// With c the cotangent that row t+1 hands back (behind a sequence's last row dfinal):
//     d = dout_t + c,  dx = d (or (1 - a) d),  dg = d a h_{t-1} (0 below the bound), or
//     d (h_{t-1} - x) a (1 - a),  c <- a d,  and dinitial is what the first row hands back.
// The same chain run from the last row to the first; h is the forward's output, so
// h_{t-1} carries the rounding of its type (half a step, as the gradient itself does), which
// saves the forward's recomputation and the reading of x in the log form.
template <typename T, bool VEC, bool SIG, int S>
__global__ void __launch_bounds__(kScanThreads, 2) scan_bwd_kernel(const __grid_constant__ ScanBwdParams p) {
    constexpr int L = kScanWarps * S;
    __shared__ ScanShared<L> sm;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int link, tile;  // place in the chain; rows run the other way
    take_item(sm, p.chain, link, tile);
    const int chunk = p.chain.chunks - 1 - link, block = kScanWarps - 1 - warp;
    const int row0 = chunk * L, wrow = row0 + block * S, R = p.span.R, D = p.D;

    Raw4<T> dr[S], gr[S], hr[S], xr[SIG ? S : 1];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int row = wrow + s;
        const bool ok = row < R;
        dr[s] = load_row<T, VEC>(static_cast<const T *>(p.dout) + (long long)row * p.dout_stride, tile, lane, D, ok);
        gr[s] = load_row<T, VEC>(static_cast<const T *>(p.g) + (long long)row * p.g_stride, tile, lane, D, ok);
        hr[s] = load_row<T, VEC>(static_cast<const T *>(p.h) + (long long)(row - 1) * p.h_stride, tile, lane, D, ok && row > 0);
        if (SIG) xr[s] = load_row<T, VEC>(static_cast<const T *>(p.x) + (long long)row * p.x_stride, tile, lane, D, ok);
    }
    fill_rows<L>(sm.map, p.span, row0, [&](int n) {
        if (!p.ds0) return;
        const int c1 = min(D, (tile + 1) * kTileChannels);
        for (int c = tile * kTileChannels; c < c1; ++c) p.ds0[(long long)n * D + c] = p.dsT ? p.dsT[(long long)n * D + c] : 0.f;
    });
    if (R == 0) return;
    const unsigned starts = row_bits<S>(sm.map.start + block * S, lane), ends = row_bits<S>(sm.map.end + block * S, lane);

    float A[4] = {1.f, 1.f, 1.f, 1.f}, H[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
        float cT[4];
        const bool end = ends >> s & 1;
        if (end) state_or_zero<VEC>(p.dsT, sm.map.end[block * S + s], tile, lane, D, cT);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            decay<SIG>(raw_get(gr[s], i), p.has_lb, p.lb, a, b);
            H[i] = a * (raw_get(dr[s], i) + (end ? cT[i] : H[i]));
            A[i] = end ? 0.f : A[i] * a;
        }
    }
    float c[4];
    const bool carry = sm.map.behind > row0 + L;
    const int last = min(max(sm.map.behind - 1, 0), R - 1);
    join<L>(sm, p.chain, link, tile, carry, p.chain.chunks - 1 - last / L, A, H, ends != 0, c);
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
        const int row = wrow + s;
        if (row < R) {
            float hp[4], dx[4], dg[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) hp[i] = raw_get(hr[s], i);
            if (ends >> s & 1) state_or_zero<VEC>(p.dsT, sm.map.end[block * S + s], tile, lane, D, c);
            if (starts >> s & 1) state_or_zero<VEC>(p.s0, sm.map.start[block * S + s], tile, lane, D, hp);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g = raw_get(gr[s], i), d = raw_get(dr[s], i) + c[i];
                float a, b;
                decay<SIG>(g, p.has_lb, p.lb, a, b);
                c[i] = a * d;
                if (SIG) {
                    dx[i] = b * d;
                    dg[i] = c[i] * b * (hp[i] - raw_get(xr[s], i));
                } else {
                    dx[i] = d;
                    dg[i] = p.has_lb && g < p.lb ? 0.f : c[i] * hp[i];
                }
            }
            store_row<T, VEC>(static_cast<T *>(p.dx) + (long long)row * D, tile, lane, D, dx);
            store_row<T, VEC>(static_cast<T *>(p.dg) + (long long)row * D, tile, lane, D, dg);
            if (p.ds0 && (starts >> s & 1)) store_state<VEC>(p.ds0, sm.map.start[block * S + s], tile, lane, D, c);
        }
    }
    publish_group(p.chain, link, tile, c);
}

// ---------------------------------------------------------------- single token
template <typename T, bool VEC, bool SIG>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ ScanStepParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = (p.D + kTileChannels - 1) / kTileChannels;
    const long long item = (long long)blockIdx.x * 4 + warp;
    const int n = (int)(item / tiles), tile = (int)(item - (long long)n * tiles);
    if (n >= p.N) return;
    const Raw4<T> x = load_row<T, VEC>(static_cast<const T *>(p.x) + n * p.x_stride, tile, lane, p.D, true);
    const Raw4<T> g = load_row<T, VEC>(static_cast<const T *>(p.g) + n * p.g_stride, tile, lane, p.D, true);
    float h[4];
    load_f32<VEC>(p.state + (long long)n * p.D, tile, lane, p.D, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        decay<SIG>(raw_get(g, i), p.has_lb, p.lb, a, b);
        h[i] = fmaf(a, h[i], SIG ? b * raw_get(x, i) : raw_get(x, i));
    }
    store_state<VEC>(p.state_out, n, tile, lane, p.D, h);
    store_row<T, VEC>(static_cast<T *>(p.h) + (long long)n * p.D, tile, lane, p.D, h);
}

// ---------------------------------------------------------------- host
bool vec_ok(const void *p, long long stride, size_t esz) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (4 * esz) == 0 && stride % 4 == 0);
}

// Rows a warp holds: fp32 holds half of bf16's, so that the backward's four tensors fit.
int scan_rows(bool bf16) { return kScanWarps * (bf16 ? 8 : 4); }

int tiles_of(int D) { return (D + kTileChannels - 1) / kTileChannels; }

// Chunks per group: as many as are in flight of one tile at a time, so that a wave's
// chunks wait for about one chained state. More would read maps for nothing.
int group_of(int chunks, int tiles) {
    int g = 1;
    while (g < 32 && g * tiles < 2 * 148) g *= 2;
    return g;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

size_t scan_layout(int rows, int D, bool bf16, void *ws, ScanChain *ch) {
    const int L = scan_rows(bf16);
    const int chunks = rows > L ? (rows + L - 1) / L : 1, tiles = tiles_of(D);
    const int group = group_of(chunks, tiles);
    size_t at = 0;
    char *base = static_cast<char *>(ws);
    if (ch) { ch->chunks = chunks; ch->tiles = tiles; ch->group = group; }
    if (chunks == 1) return 0;
    if (ch) { ch->status = reinterpret_cast<int *>(base); ch->ticket = reinterpret_cast<unsigned *>(base) + 1; }
    if (ch) ch->flags = reinterpret_cast<unsigned *>(base + 256);
    at = 256 + round256(sizeof(unsigned) * (size_t)chunks * tiles);
    if (ch) ch->agg = reinterpret_cast<float2 *>(base + at);
    at += round256(sizeof(float2) * (size_t)chunks * tiles * kTileChannels);
    if (ch) ch->inc = reinterpret_cast<float *>(base + at);
    at += round256(sizeof(float) * (size_t)(chunks / group) * tiles * kTileChannels);
    return at;
}

// Clears what a chain starts from: status, ticket and flags.
cudaError_t clear_chain(const ScanChain &ch, cudaStream_t st) {
    if (ch.chunks == 1) return cudaSuccess;
    return cudaMemsetAsync(ch.status, 0, 256 + sizeof(unsigned) * (size_t)ch.chunks * ch.tiles, st);
}

template <typename T, bool VEC, bool SIG> cudaError_t run_fwd(const ScanParams &p, cudaStream_t st) {
    count_launch();
    scan_fwd_kernel<T, VEC, SIG, sizeof(T) == 2 ? 8 : 4>
        <<<(unsigned)(p.chain.chunks * p.chain.tiles), kScanThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T, bool VEC, bool SIG> cudaError_t run_bwd(const ScanBwdParams &p, cudaStream_t st) {
    count_launch();
    scan_bwd_kernel<T, VEC, SIG, sizeof(T) == 2 ? 8 : 4>
        <<<(unsigned)(p.chain.chunks * p.chain.tiles), kScanThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T, bool VEC, bool SIG> cudaError_t run_step(const ScanStepParams &p, cudaStream_t st) {
    const long long items = (long long)p.N * tiles_of(p.D);
    count_launch();
    scan_step_kernel<T, VEC, SIG><<<(unsigned)((items + 3) / 4), 128, 0, st>>>(p);
    return cudaGetLastError();
}

// Runs F<T, VEC, SIG> for the types of a call.
#define KDA_SCAN_PICK(F, p, bf16, vec, sig, st)                                                       \
    (bf16 ? (vec ? (sig ? F<__nv_bfloat16, true, true>(p, st) : F<__nv_bfloat16, true, false>(p, st))   \
                 : (sig ? F<__nv_bfloat16, false, true>(p, st) : F<__nv_bfloat16, false, false>(p, st))) \
          : (vec ? (sig ? F<float, true, true>(p, st) : F<float, true, false>(p, st))                   \
                 : (sig ? F<float, false, true>(p, st) : F<float, false, false>(p, st))))

}  // namespace

size_t scan_workspace_bytes(int rows, int D, bool bf16, bool) { return scan_layout(rows, D, bf16, nullptr, nullptr); }

cudaError_t launch_scan(ScanParams p, bool bf16, bool sigmoid, void *workspace, cudaStream_t st) {
    const int stall = p.chain.stall;
    scan_layout(p.span.R, p.D, bf16, workspace, &p.chain);
    p.chain.stall = stall;
    if ((long long)p.chain.chunks * p.chain.tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t e = clear_chain(p.chain, st);
    if (e != cudaSuccess) return e;
    const size_t esz = bf16 ? 2 : 4;
    const bool vec = p.D % 4 == 0 && vec_ok(p.x, p.x_stride, esz) && vec_ok(p.g, p.g_stride, esz) &&
                     vec_ok(p.h, p.D, esz) && vec_ok(p.s0, p.D, 4) && vec_ok(p.sT, p.D, 4);
    return KDA_SCAN_PICK(run_fwd, p, bf16, vec, sigmoid, st);
}

cudaError_t launch_scan_bwd(ScanBwdParams p, bool bf16, bool sigmoid, void *workspace, cudaStream_t st) {
    const int stall = p.chain.stall;
    scan_layout(p.span.R, p.D, bf16, workspace, &p.chain);
    p.chain.stall = stall;
    if ((long long)p.chain.chunks * p.chain.tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t e = clear_chain(p.chain, st);
    if (e != cudaSuccess) return e;
    const size_t esz = bf16 ? 2 : 4;
    const bool vec = p.D % 4 == 0 && vec_ok(p.x, p.x_stride, esz) && vec_ok(p.g, p.g_stride, esz) &&
                     vec_ok(p.h, p.h_stride, esz) && vec_ok(p.dout, p.dout_stride, esz) && vec_ok(p.dx, p.D, esz) &&
                     vec_ok(p.dg, p.D, esz) && vec_ok(p.s0, p.D, 4) && vec_ok(p.dsT, p.D, 4) && vec_ok(p.ds0, p.D, 4);
    return KDA_SCAN_PICK(run_bwd, p, bf16, vec, sigmoid, st);
}

cudaError_t launch_scan_step(const ScanStepParams &p, bool bf16, bool sigmoid, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4;
    const bool vec = p.D % 4 == 0 && vec_ok(p.x, p.x_stride, esz) && vec_ok(p.g, p.g_stride, esz) &&
                     vec_ok(p.h, p.D, esz) && vec_ok(p.state, p.D, 4) && vec_ok(p.state_out, p.D, 4);
    return KDA_SCAN_PICK(run_step, p, bf16, vec, sigmoid, st);
}

}  // namespace kda

// Walkers: how the operators that run along time over packed [rows, channels] tensors cut
// and read them. A walker is one warp (and one CTA) that walks 32 LB bytes of channels (LB =
// 4 or 8 bytes a lane: 64 or 128 channels in bf16, half of that in fp32) down a piece of the
// rows, with what it carries in registers. Asynchronous copies run stages of rows ahead of
// it into a ring in its own shared memory, so no barrier and no other warp is involved,
// every element is read once, and the walkers of an SM keep some 170 KB of reads in flight
// between them.
#pragma once

#include <type_traits>

#include "kda_common.cuh"
#include "kda_stage.cuh"

namespace kda {

// Sequences packed along the rows: sequence n is rows cu[n] .. cu[n+1]-1, or, without
// offsets, rows n*T .. (n+1)*T-1. R rows in all.
struct RowSpan {
    const int32_t *cu;
    int T, N, R;
};

// Channels of a lane, and of a walker.
template <typename T, int LB> constexpr int lane_channels() { return LB / (int)sizeof(T); }
template <typename T, int LB> constexpr int walk_channels() { return 32 * lane_channels<T, LB>(); }

// ---------------------------------------------------------------- passes of a call
// The pass that joins a backward pass's partial sums is queued while that one runs: its CTAs
// come up as SMs empty and wait for the sums, all of them, so that its end is the end of both
// (1 us a call). The scan's passes follow one another plainly: a walk whose CTAs come up
// early crowds the first SMs to empty (131072 x 257: 244 us against 211).
__device__ __forceinline__ void let_next_pass_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last_pass() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P>
cudaError_t launch_next_pass(void (*kernel)(P...), unsigned grid, unsigned threads, cudaStream_t st,
                        typename std::common_type<P>::type... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(threads);
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    count_launch();
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args...);
    return e != cudaSuccess ? cudaGetLastError() : e;
}

// Launches a walker, one warp, for each piece and channel unit.
template <typename P> cudaError_t run_walk(void (*kernel)(P), const P &p, int pieces, int units, int ring_bytes, cudaStream_t st) {
    const long long grid = (long long)pieces * units;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    count_launch();
    kernel<<<(unsigned)grid, 32, ring_bytes, st>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- arithmetic
// The SFU's exponential (off by 2 steps) and reciprocal (1 step), for bf16 results.
__device__ __forceinline__ float ex2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;
// sigmoid, by the SFU where the result is rounded to bf16 (2 + 1 steps off).
template <typename T> __device__ __forceinline__ float sig(float x) {
    return sizeof(T) == 2 ? rcp_fast(1.f + ex2_fast(-kLog2e * x)) : 1.f / (1.f + expf(-x));
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(p);
}

// d = a b + c, d = a b, d = a + b of a lane's channels: one instruction for two.
__device__ __forceinline__ void pair_fma(const float *a, const float *b, const float *c, float *d) {
    asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rc, ra, rb, rc;\n\tmov.b64 {%0, %1}, rc;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void pair_mul(const float *a, const float *b, float *d) {
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
__device__ __forceinline__ void pair_add(const float *a, const float *b, float *d) {
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
template <int W> __device__ __forceinline__ void vfma(const float (&a)[W], const float (&b)[W], const float (&c)[W], float (&d)[W]) {
    if constexpr (W == 1) {
        d[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 2) pair_fma(a + i, b + i, c + i, d + i);
    }
}
template <int W> __device__ __forceinline__ void vmul(const float (&a)[W], const float (&b)[W], float (&d)[W]) {
    if constexpr (W == 1) {
        d[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 2) pair_mul(a + i, b + i, d + i);
    }
}
template <int W> __device__ __forceinline__ void vadd(const float (&a)[W], const float (&b)[W], float (&d)[W]) {
    if constexpr (W == 1) {
        d[0] = a[0] + b[0];
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 2) pair_add(a + i, b + i, d + i);
    }
}
template <int W> __device__ __forceinline__ void vset(float (&d)[W], float v) {
#pragma unroll
    for (int i = 0; i < W; ++i) d[i] = v;
}

// The sum of column `col` over `slices` rows of `cols` partial sums, by a CTA of 32 warps:
// each warp adds its share in order, then the warps' sums are added in order. The result is
// the first warp's, whose lanes hold 32 neighbouring columns.
__device__ __forceinline__ float slice_sum(const float *partial, int slices, long long cols, long long col) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float s = 0.f;
    if (col < cols) {
#pragma unroll 8
        for (int j = warp; j < slices; j += 32) s += partial[j * cols + col];
    }
    red[warp][lane] = s;
    __syncthreads();
    float v = 0.f;
    if (warp == 0)
#pragma unroll
        for (int j = 0; j < 32; ++j) v += red[j][lane];
    return v;
}

// ---------------------------------------------------------------- staged rows
// A tensor as a walker reads it: its first channel of row 0, the bytes between rows, and
// where the tensor begins and ends.
struct WalkTensor {
    const char *at;
    long long stride;
    const char *begin, *end;
};
template <typename T>
__device__ __forceinline__ WalkTensor walk_tensor(const void *base, long long stride, int c0, int C, int R) {
    const char *b = static_cast<const char *>(base);
    return {b + (long long)c0 * sizeof(T), stride * (long long)sizeof(T), b,
            b + ((long long)(R - 1) * stride + C) * (long long)sizeof(T)};
}

// The lane's channels of a row as stored, and unpacked.
template <int LB> struct Raw {
    uint32_t w[LB / 4];
};
template <typename T, int LB> __device__ __forceinline__ void unpack(const Raw<LB> &r, float (&v)[lane_channels<T, LB>()]) {
#pragma unroll
    for (int i = 0; i < LB / 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            v[i] = __uint_as_float(r.w[i]);
        } else {
            v[2 * i] = __uint_as_float(r.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
        }
    }
}

// How rows are accessed: by G bytes at a time, G the largest of 16, 8, 4 and 2 that divides
// the base, the row stride and the row's length of all the tensors of a call.
struct RowAccess {
    unsigned long long bits = 0;
    void rows(const void *p, long long stride, long long C, size_t esz) {
        if (p) bits |= reinterpret_cast<uintptr_t>(p) | (unsigned long long)stride * esz | (unsigned long long)C * esz;
    }
    int g() const { return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2; }
};

// The ring of a walker: STAGES stages of S rows of N tensors. Rows of 16-, 8- or 4-byte
// aligned elements are copied to where a lane reads its LB bytes at once. Rows of single
// bf16 elements (G = 2: odd widths) are copied with the 16-byte words that hold them -- those
// that reach beyond the tensor element by element -- and read at their offset in those.
template <typename T, int G, int LB, int S, int N, int STAGES> struct Ring {
    static constexpr int W = lane_channels<T, LB>(), ROW = 32 * LB;
    static constexpr bool WHOLE = G > 2;  // rows are copied to where lanes read them
    static constexpr int PITCH = WHOLE ? ROW : ROW + 16, PART = S * PITCH, BYTES = STAGES * N * PART;
    char *base;
    WalkTensor t[N];
    int width;  // bytes of a row that are the walker's
    int lane;
    const char *src[N];  // where the lane's next copies begin

    // A lane's first copy of a stage: its row in the stage, its byte in the row.
    static constexpr int PER = ROW / G;  // copies of a row
    static constexpr int ROWS = PER < 32 ? 32 / PER : 1, ROUNDS = PER < 32 ? 1 : PER / 32;
    static_assert(!WHOLE || S % ROWS == 0, "whole rounds");
    __device__ __forceinline__ int lane_row() const { return PER < 32 ? lane / PER : 0; }
    __device__ __forceinline__ int lane_byte() const { return (PER < 32 ? lane % PER : lane) * G; }
    // Where it reads from. In the last, partly filled unit lanes beyond the row copy its first
    // bytes, to places that nothing is written from: predicates on every copy instead cost
    // 31744 x 12288 bf16 537 us against 511, a loop over rows 8192 x 2000 backward 58 against 49.
    // Rows of two narrow copies a lane (MASKED) do take predicates: 131072 x 257 fp32 211 us,
    // where copying the first bytes 64 times over takes 457.
    static constexpr bool MASKED = ROUNDS > 1;
    __device__ __forceinline__ int lane_from() const { return MASKED || lane_byte() < width ? lane_byte() : 0; }

    // The next stage of tensor i to be loaded is the one that begins at `row`.
    __device__ __forceinline__ void begin(int i, int row) {
        src[i] = t[i].at + (long long)row * t[i].stride;
        if (WHOLE) src[i] += lane_row() * t[i].stride + lane_from();
    }

    template <int B> static __device__ __forceinline__ void copy(unsigned to, const char *from) {
        if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(B) : "memory");
    }

    // Starts the copies of the next stage of tensor i, rows row .. row+S-1, into `slot`: those
    // in [lo, hi). DIR: whether the stage after it lies behind (1) or before it (-1).
    template <int DIR> __device__ __forceinline__ void load(int slot, int i, int row, int lo, int hi) {
        const char *from = src[i];
        src[i] += DIR * S * t[i].stride;
        char *to = base + (slot * N + i) * PART;
        const bool inner = row >= lo && row + S <= hi;
        if constexpr (WHOLE) {
            const int lr = lane_row(), lc = lane_byte();
            const unsigned d = (unsigned)__cvta_generic_to_shared(to + lr * PITCH + lc);
            const long long step = ROWS * t[i].stride;
            if (inner) {
#pragma unroll
                for (int k = 0; k < S; k += ROWS, from += step)
#pragma unroll
                    for (int j = 0; j < ROUNDS; ++j)
                        if (!MASKED || lc + j * 32 * G < width) copy<G>(d + k * PITCH + j * 32 * G, from + j * 32 * G);
                return;
            }
#pragma unroll 1
            for (int k = 0; k < S; k += ROWS, from += step) {
                const int r = row + lr + k;
                if (r >= lo && r < hi)
#pragma unroll
                    for (int j = 0; j < ROUNDS; ++j)
                        if (!MASKED || lc + j * 32 * G < width) copy<G>(d + k * PITCH + j * 32 * G, from + j * 32 * G);
            }
        } else {
            constexpr int WORDS = PITCH / 16, COUNT = S * WORDS;
            // words near the tensor's first and last rows may reach beyond it
            const bool plain = inner && from - 14 >= t[i].begin && from + (S - 1) * t[i].stride + width + 14 <= t[i].end;
            if (plain) {
#pragma unroll
                for (int q = 0; q < (COUNT + 31) / 32; ++q) {
                    const int x = q * 32 + lane, k = x / WORDS, j = x - k * WORDS;
                    const char *a = from + k * t[i].stride;
                    const int off = (int)((uint32_t)reinterpret_cast<uintptr_t>(a) & 15u);
                    if (x < COUNT && 16 * j - off < width) copy<16>((unsigned)__cvta_generic_to_shared(to + x * 16), a - off + 16 * j);
                }
                return;
            }
#pragma unroll 1
            for (int x = lane; x < COUNT; x += 32) {
                const int k = x / WORDS, j = x - k * WORDS, r = row + k;
                if (r < lo || r >= hi) continue;
                const char *a = from + k * t[i].stride;
                const int off = (int)((uint32_t)reinterpret_cast<uintptr_t>(a) & 15u);
                const char *w = a - off + 16 * j;
                if (16 * j - off >= width) continue;
                if (w >= t[i].begin && w + 16 <= t[i].end) {
                    copy<16>((unsigned)__cvta_generic_to_shared(to + x * 16), w);
                } else {
                    for (int e = 0; e < 16; e += (int)sizeof(T))
                        if (16 * j - off + e >= 0 && 16 * j - off + e < width)
                            *reinterpret_cast<T *>(to + x * 16 + e) = *reinterpret_cast<const T *>(w + e);
                }
            }
        }
    }
    // The lane's channels of row r, the s-th of stage `slot`.
    __device__ __forceinline__ Raw<LB> raw(int slot, int i, int s, int r) const {
        const char *p = base + (slot * N + i) * PART + s * PITCH + lane * LB;
        Raw<LB> q;
        if constexpr (WHOLE) {
            if constexpr (LB == 4) q.w[0] = *reinterpret_cast<const uint32_t *>(p);
            else reinterpret_cast<uint2 &>(q) = *reinterpret_cast<const uint2 *>(p);
        } else {
            const uint32_t shift = ((uint32_t)reinterpret_cast<uintptr_t>(t[i].at) + (uint32_t)r * (uint32_t)t[i].stride) & 15u;
            const uint32_t *w = reinterpret_cast<const uint32_t *>(p + (shift & 12u));
#pragma unroll
            for (int j = 0; j < LB / 4; ++j) q.w[j] = __funnelshift_r(w[j], w[j + 1], shift * 8u & 16u);
        }
        return q;
    }
    __device__ __forceinline__ void get(int slot, int i, int s, int r, float (&v)[W]) const { unpack<T, LB>(raw(slot, i, s, r), v); }
};

// Stores the lane's channels, from c on, of an output row (the whole warp takes part).
template <int G, int W> __device__ __forceinline__ void put_row(float *row, int c, int C, int, const float (&v)[W]) {
    if constexpr (G >= 8 && W == 2) {
        if (c < C) *reinterpret_cast<float2 *>(row + c) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (c + i < C) row[c + i] = v[i];
    }
}
template <int G, int W> __device__ __forceinline__ void put_row(__nv_bfloat16 *row, int c, int C, int lane, const float (&v)[W]) {
    if constexpr (G >= 8 && W == 4) {
        if (c < C) *reinterpret_cast<uint2 *>(row + c) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else if constexpr (G >= 4) {
#pragma unroll
        for (int i = 0; i < W; i += 2)
            if (c + i < C) *reinterpret_cast<uint32_t *>(row + c + i) = pack_bf16(v[i], v[i + 1]);
    } else {
        // where the row begins in the middle of a word, words pair a lane's last channel with the next lane's first
        const bool odd = reinterpret_cast<uintptr_t>(row) & 2;
        float x[W];
        x[0] = __shfl_up_sync(0xffffffffu, v[W - 1], 1);
#pragma unroll
        for (int i = W - 1; i > 0; --i) x[i] = odd ? v[i - 1] : v[i];
        if (!odd) x[0] = v[0];
        const int at = odd ? c - 1 : c;
        __nv_bfloat16 *p = row + at;
        const bool edge = odd && lane == 0;  // its first word is shared with the tile before
#pragma unroll
        for (int i = 0; i < W; i += 2) {
            const uint32_t q = pack_bf16(x[i], x[i + 1]);
            if (at + i + 1 < C && !(edge && i == 0)) *reinterpret_cast<uint32_t *>(p + i) = q;
            else if (at + i < C && !(edge && i == 0)) *reinterpret_cast<uint16_t *>(p + i) = (uint16_t)q;
        }
        if (edge && c < C) row[c] = __float2bfloat16_rn(v[0]);
        if (odd && lane == 31 && c + W - 1 < C) row[c + W - 1] = __float2bfloat16_rn(v[W - 1]);
    }
}

// ---------------------------------------------------------------- rows and sequences
// First i in [0, n] with a[i] >= v of n non-decreasing values, by one warp: 32 probes a
// round. Reads nothing outside the n values, and ends, whatever they hold.
__device__ __forceinline__ int warp_lower_bound(const int32_t *a, int n, int v, int lane) {
    int lo = 0, hi = n;
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const int below = __popc(__ballot_sync(0xffffffffu, i < hi && a[i] < v));
        if (below == 0) break;
        hi = min(hi, lo + below * step);
        lo = lo + (below - 1) * step + 1;
    }
    return min(lo, n);
}

// A sequence and its rows.
struct Seq {
    int n, start, end;
};

// The sequence that holds `row` < R, by the whole warp. Whatever cu holds, start <= row < end.
__device__ __forceinline__ Seq seq_of(const RowSpan &sp, int row, int lane) {
    Seq q;
    if (sp.cu) {
        q.n = min(max(warp_lower_bound(sp.cu, sp.N + 1, row + 1, lane) - 1, 0), sp.N - 1);
        q.start = min(max(sp.cu[q.n], 0), row);
        q.end = min(max(sp.cu[q.n + 1], row + 1), sp.R);
    } else {
        q.n = row / sp.T;
        q.start = q.n * sp.T;
        q.end = q.start + sp.T;
    }
    return q;
}

// Pieces share out the empty sequences, whose states of M values a channel go from one
// side to the other: channels c .. c+W-1 of each.
template <int W>
__device__ __forceinline__ void hand_through(const RowSpan &sp, int piece, int pieces, int lane, int c, int C, int M, float *to,
                                             const float *from) {
    if (!to || (!sp.cu && sp.T > 0)) return;
    for (long long n0 = (long long)piece * 32; n0 < sp.N; n0 += (long long)pieces * 32) {
        const int n = (int)n0 + lane;
        unsigned empty = __ballot_sync(0xffffffffu, n < sp.N && (!sp.cu || sp.cu[n + 1] <= sp.cu[n]));
        while (empty) {
            const long long at = ((n0 + __ffs(empty) - 1) * C + c) * M;
            empty &= empty - 1;
            for (int i = 0; i < W * M; ++i)
                if (c + i / M < C) to[at + i] = from ? from[at + i] : 0.f;
        }
    }
}

}  // namespace kda

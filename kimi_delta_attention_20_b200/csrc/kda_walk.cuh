// Walkers: how the operators that run along time over packed [rows, channels] tensors cut
// and read them. A walker is one warp (and one CTA) that walks 128 bytes of channels -- 64
// in bf16, 32 in fp32, 4 bytes a lane -- down a piece of the rows, with what it carries in
// registers. Asynchronous copies run stages of 16 rows ahead of it into a ring in its own
// shared memory, so no barrier and no other warp is involved, every element is read once,
// and the walkers of an SM keep some 170 KB of reads in flight between them.
#pragma once

#include "kda_common.cuh"
#include "kda_stage.cuh"

namespace kda {

// Sequences packed along the rows: sequence n is rows cu[n] .. cu[n+1]-1, or, without
// offsets, rows n*T .. (n+1)*T-1. R rows in all.
struct RowSpan {
    const int32_t *cu;
    int T, N, R;
};

constexpr int kStageRows = 16;
constexpr int kWalkBytes = 128;

// Channels of a walker, and of a lane.
template <typename T> constexpr int walk_channels() { return kWalkBytes / (int)sizeof(T); }
template <typename T> constexpr int lane_channels() { return 4 / (int)sizeof(T); }

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
__device__ __forceinline__ void vfma(const float (&a)[1], const float (&b)[1], const float (&c)[1], float (&d)[1]) { d[0] = fmaf(a[0], b[0], c[0]); }
__device__ __forceinline__ void vmul(const float (&a)[1], const float (&b)[1], float (&d)[1]) { d[0] = a[0] * b[0]; }
__device__ __forceinline__ void vadd(const float (&a)[1], const float (&b)[1], float (&d)[1]) { d[0] = a[0] + b[0]; }
__device__ __forceinline__ void vfma(const float (&a)[2], const float (&b)[2], const float (&c)[2], float (&d)[2]) {
    asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rc, ra, rb, rc;\n\tmov.b64 {%0, %1}, rc;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void vmul(const float (&a)[2], const float (&b)[2], float (&d)[2]) {
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
__device__ __forceinline__ void vadd(const float (&a)[2], const float (&b)[2], float (&d)[2]) {
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
template <int W> __device__ __forceinline__ void vset(float (&d)[W], float v) {
#pragma unroll
    for (int i = 0; i < W; ++i) d[i] = v;
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

// The ring of a walker: STAGES stages of 16 rows of N tensors. AL: rows and base are
// 16-byte aligned. Otherwise a row is copied with the 16-byte words that hold it (those
// that reach beyond the tensor element by element) and read at its offset in them, so odd
// widths and odd slices move the same bytes in almost as few instructions.
template <typename T, bool AL, int N, int STAGES> struct Ring {
    static constexpr int W = lane_channels<T>();
    static constexpr int PITCH = AL ? kWalkBytes : kWalkBytes + 16, PART = kStageRows * PITCH, BYTES = STAGES * N * PART;
    static constexpr int WORDS = PITCH / 16;
    char *base;
    WalkTensor t[N];
    int width;  // bytes of a row that are the walker's
    int lane;

    // Starts the copies of rows row .. row+15 of tensor i into stage `slot`: those in [lo, hi).
    __device__ __forceinline__ void load(int slot, int i, int row, int lo, int hi) const {
        char *to = base + (slot * N + i) * PART;
        if (AL) {
            const int lr = lane >> 3, lc = (lane & 7) * 16;
            const char *src = t[i].at + (long long)(row + lr) * t[i].stride + lc;
            unsigned d = (unsigned)__cvta_generic_to_shared(to + lr * PITCH + lc);
#pragma unroll
            for (int k = 0; k < kStageRows; k += 4) {
                const int r = row + lr + k;
                if (r >= lo && r < hi && lc < width)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + k * PITCH), "l"(src + k * t[i].stride) : "memory");
            }
            return;
        }
#pragma unroll
        for (int q = 0; q < (kStageRows * WORDS + 31) / 32; ++q) {
            const int x = q * 32 + lane, k = x / WORDS, j = x - k * WORDS, r = row + k;
            if (k < kStageRows && r >= lo && r < hi) {
                const char *a = t[i].at + (long long)r * t[i].stride;
                const char *w = a - (reinterpret_cast<uintptr_t>(a) & 15) + 16 * j;
                if (w < a + width) {
                    if (w >= t[i].begin && w + 16 <= t[i].end) {
                        const unsigned d = (unsigned)__cvta_generic_to_shared(to + k * PITCH + 16 * j);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(w) : "memory");
                    } else {
                        for (int b = 0; b < 16; b += (int)sizeof(T))
                            if (w + b >= a && w + b < a + width)
                                *reinterpret_cast<T *>(to + k * PITCH + 16 * j + b) = *reinterpret_cast<const T *>(w + b);
                    }
                }
            }
        }
    }
    // The lane's channels of row r, the s-th of stage `slot`.
    __device__ __forceinline__ void get(int slot, int i, int s, int r, float (&v)[W]) const {
        const char *p = base + (slot * N + i) * PART + s * PITCH + lane * 4;
        uint32_t q;
        if (AL) {
            q = *reinterpret_cast<const uint32_t *>(p);
        } else {
            const uint32_t shift = ((uint32_t)reinterpret_cast<uintptr_t>(t[i].at) + (uint32_t)r * (uint32_t)t[i].stride) & 15u;
            const uint32_t *w = reinterpret_cast<const uint32_t *>(p + (shift & 12u));
            q = w[0];
            if (sizeof(T) == 2) q = __funnelshift_r(q, w[1], (shift & 2u) * 8u);
        }
        if constexpr (W == 1) {
            v[0] = __uint_as_float(q);
        } else {
            v[0] = __uint_as_float(q << 16);
            v[1] = __uint_as_float(q & 0xffff0000u);
        }
    }
};

// Stores the lane's channels, from c on, of an output row (the whole warp takes part).
template <bool AL> __device__ __forceinline__ void put_row(float *row, int c, int C, int, const float (&v)[1]) {
    if (c < C) row[c] = v[0];
}
template <bool AL> __device__ __forceinline__ void put_row(__nv_bfloat16 *row, int c, int C, int lane, const float (&v)[2]) {
    if (AL) {
        if (c < C) *reinterpret_cast<uint32_t *>(row + c) = pack_bf16(v[0], v[1]);
        return;
    }
    if (reinterpret_cast<uintptr_t>(row) & 2) {
        // the row begins in the middle of a word: words pair a lane's second channel with the next lane's first
        const float before = __shfl_up_sync(0xffffffffu, v[1], 1);
        if (lane == 0) {
            if (c < C) row[c] = __float2bfloat16_rn(v[0]);
        } else if (c < C) {
            *reinterpret_cast<uint32_t *>(row + c - 1) = pack_bf16(before, v[0]);
        } else if (c - 1 < C) {
            row[c - 1] = __float2bfloat16_rn(before);
        }
        if (lane == 31 && c + 1 < C) row[c + 1] = __float2bfloat16_rn(v[1]);
    } else if (c + 1 < C) {
        *reinterpret_cast<uint32_t *>(row + c) = pack_bf16(v[0], v[1]);
    } else if (c < C) {
        row[c] = __float2bfloat16_rn(v[0]);
    }
}

// Whether all the tensors of a call have 16-byte aligned rows.
struct Aligned {
    bool ok = true;
    void rows(const void *p, long long stride, long long C, size_t esz) {
        if (p && ((reinterpret_cast<uintptr_t>(p) | (unsigned long long)stride * esz | (unsigned long long)C * esz) & 15)) ok = false;
    }
};

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

// Packed rows: what the operators that walk [rows, channels] tensors along the token
// axis share -- four channels per lane, and the map from packed rows to sequences.
#pragma once

#include "kda_common.cuh"

namespace kda {

// Sequences packed along the rows: sequence n is rows cu[n] .. cu[n+1]-1, or, without
// offsets, rows n*T .. (n+1)*T-1. R rows in all.
struct RowSpan {
    const int32_t *cu;
    int T, N, R;
};

// ---------------------------------------------------------------- four channels of a row
constexpr int kLaneChannels = 4;
constexpr int kTileChannels = 32 * kLaneChannels;  // channels of a warp

template <typename T> struct Raw4;
template <> struct Raw4<float> { float v[4]; };
template <> struct Raw4<__nv_bfloat16> { uint32_t v[2]; };

__device__ __forceinline__ float raw_get(const Raw4<float> &r, int i) { return r.v[i]; }
__device__ __forceinline__ float raw_get(const Raw4<__nv_bfloat16> &r, int i) {
    return __uint_as_float(i & 1 ? r.v[i >> 1] & 0xffff0000u : r.v[i >> 1] << 16);
}

// Channel i (0..3) of a lane: four neighbours where rows are read as vectors, else 32
// apart, so that the single loads of a warp touch neighbours.
template <bool VEC> __device__ __forceinline__ int lane_channel(int tile, int lane, int i) {
    return tile * kTileChannels + (VEC ? lane * 4 + i : i * 32 + lane);
}

// The lane's four channels of the row at `row` (channels beyond C read as zero). VEC: the
// row is aligned to four elements and C is a multiple of four.
template <typename T, bool VEC>
__device__ __forceinline__ Raw4<T> load_row(const T *row, int tile, int lane, int C, bool ok) {
    Raw4<T> r;
    if (VEC) {
        const int c = lane_channel<true>(tile, lane, 0);
        if (sizeof(T) == 2) {
            const uint2 q = ok && c < C ? *reinterpret_cast<const uint2 *>(row + c) : make_uint2(0u, 0u);
            reinterpret_cast<uint2 &>(r) = q;
        } else {
            const float4 q = ok && c < C ? *reinterpret_cast<const float4 *>(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            reinterpret_cast<float4 &>(r) = q;
        }
        return r;
    }
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane_channel<false>(tile, lane, i);
        q[i] = 0u;
        if (ok && c < C) {
            if (sizeof(T) == 2) q[i] = reinterpret_cast<const unsigned short *>(row)[c];
            else q[i] = reinterpret_cast<const uint32_t *>(row)[c];
        }
    }
    if (sizeof(T) == 2) {
        reinterpret_cast<uint2 &>(r) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    } else {
        reinterpret_cast<uint4 &>(r) = make_uint4(q[0], q[1], q[2], q[3]);
    }
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(p);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_row(T *row, int tile, int lane, int C, const float (&v)[4]) {
    if (VEC) {
        const int c = lane_channel<true>(tile, lane, 0);
        if (c >= C) return;
        if (sizeof(T) == 2)
            *reinterpret_cast<uint2 *>(row + c) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else
            *reinterpret_cast<float4 *>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane_channel<false>(tile, lane, i);
        if (c < C) row[c] = from_f32<T>(v[i]);
    }
}

template <bool VEC>
__device__ __forceinline__ void load_f32(const float *row, int tile, int lane, int C, float (&v)[4]) {
    const Raw4<float> r = load_row<float, VEC>(row, tile, lane, C, true);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r.v[i];
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

// The sequences of L rows from row0 on, in shared memory: for each row the sequence that
// starts (ends) there or -1, and for the first row the first row of its sequence and
// which it is, for the last row the row behind its sequence.
template <int L> struct RowMap {
    int start[L], end[L];
    int first, first_seq, behind;
    int lo, hi;
};

// Fills the map with all threads of the CTA (at least two warps and L threads); ends with
// a barrier. `empty(n)` is called, by one thread, for each empty sequence that lies at
// these rows (behind the last row too, where row0 + L reaches the end).
template <int L, typename Empty>
__device__ __forceinline__ void fill_rows(RowMap<L> &m, const RowSpan &p, int row0, Empty empty) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!p.cu) {
        if (tid < L) {
            const int r = row0 + tid, n = p.T > 0 ? r / p.T : 0, off = r - n * p.T;
            const bool in = r < p.R;
            m.start[tid] = in && off == 0 ? n : -1;
            m.end[tid] = in && off == p.T - 1 ? n : -1;
            if (tid == 0) { m.first = r - off; m.first_seq = n; }
            if (tid == L - 1) m.behind = r - off + p.T;
        }
        if (p.T == 0 && row0 == 0)
            for (int n = tid; n < p.N; n += blockDim.x) empty(n);
        __syncthreads();
        return;
    }
    if (warp == 0) {
        const int lo = warp_lower_bound(p.cu, p.N + 1, row0, lane);
        if (lane == 0) m.lo = lo;
    } else if (warp == 1) {
        const int hi = row0 + L >= p.R ? p.N : warp_lower_bound(p.cu, p.N + 1, row0 + L, lane);
        if (lane == 0) m.hi = hi;
    }
    if (tid < L) { m.start[tid] = -1; m.end[tid] = -1; }
    __syncthreads();
    const int lo = m.lo, hi = min(m.hi, p.N);
    if (tid == 0) {
        // lo: the first sequence that starts at row0 or later
        const bool at = lo <= p.N && p.cu[min(lo, p.N)] == row0;
        const int n = at ? lo : max(lo - 1, 0);
        m.first = at ? row0 : min(max(p.cu[n], 0), row0);
        m.first_seq = min(n, p.N - 1);
        m.behind = p.cu[hi];
    }
    for (int n = max(lo - 1, 0) + tid; n < hi; n += blockDim.x) {
        const int s = p.cu[n], e = p.cu[n + 1];
        if (e > s) {
            if (s >= row0 && s < row0 + L) m.start[s - row0] = n;
            if (e > row0 && e <= row0 + L) m.end[e - 1 - row0] = n;
        } else if (s >= row0) {
            empty(n);
        }
    }
    __syncthreads();
}

}  // namespace kda

// rows.hpp -- device helpers of the operators that work on token rows
// (convolution, scan, norms): wide row accesses, activations, sums over a
// group of threads, and the map from a workgroup's number to a tile of a
// packed sequence.
#pragma once

#include <hip/hip_runtime.h>

#include "launch.hpp"
#include "tile.hpp"

namespace gdnq {

// The workgroup's number in a grid of grid_of() that is nx wide (an argument of
// the kernel's own, read with the others).
__device__ __forceinline__ unsigned block_id(unsigned nx)
{
    return __builtin_amdgcn_workgroup_id_y() * nx + __builtin_amdgcn_workgroup_id_x();
}

// V consecutive io-dtype values, as one access of V elements (V = 1, or the
// 16 bytes of 8 bf16 / 4 fp32 values).
template <bool BF16, int V>
struct Pack {
    static_assert(V == 1 || V == (BF16 ? 8 : 4), "one element or 16 bytes");
    using elem = std::conditional_t<BF16, uint16_t, float>;
    using raw = std::conditional_t<V == 1, elem, uint4>;

    __device__ __forceinline__ static raw load(const void *base, size_t off)
    {
        return *reinterpret_cast<const raw *>(reinterpret_cast<const elem *>(base) + off);
    }

    __device__ __forceinline__ static void widen(const raw &r, float (&out)[V])
    {
        if constexpr (V == 1 && BF16) out[0] = bf16_to_f32(r);
        else if constexpr (V == 1) out[0] = r;
        else {
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if constexpr (BF16) {
                    out[2 * i] = __uint_as_float(w[i] << 16);
                    out[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                } else
                    out[i] = __uint_as_float(w[i]);
            }
        }
    }

    // rounded to nearest even
    __device__ __forceinline__ static raw narrow(const float (&v)[V])
    {
        if constexpr (V == 1 && BF16) return f32_to_bf16(v[0]);
        else if constexpr (V == 1) return v[0];
        else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if constexpr (BF16) {
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    const bf16x2 p = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
                    w[i] = __builtin_bit_cast(uint32_t, p);
                } else
                    w[i] = __float_as_uint(v[i]);
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
    }

    __device__ __forceinline__ static void store(void *base, size_t off, const raw &r)
    {
        *reinterpret_cast<raw *>(reinterpret_cast<elem *>(base) + off) = r;
    }
};

template <bool BF16, int V>
__device__ __forceinline__ void load_vec(const void *base, size_t off, float (&out)[V])
{
    Pack<BF16, V>::widen(Pack<BF16, V>::load(base, off), out);
}

template <bool BF16, int V>
__device__ __forceinline__ void store_vec(void *base, size_t off, const float (&v)[V])
{
    Pack<BF16, V>::store(base, off, Pack<BF16, V>::narrow(v));
}

// V fp32 values of a weight row (16-byte aligned where V > 1)
template <int V>
__device__ __forceinline__ void load_weights(const float *p, float (&out)[V])
{
    if constexpr (V == 1) out[0] = p[0];
    else
#pragma unroll
        for (int i = 0; i < V / 4; i++) {
            const float4 a = reinterpret_cast<const float4 *>(p)[i];
            out[4 * i] = a.x; out[4 * i + 1] = a.y; out[4 * i + 2] = a.z; out[4 * i + 3] = a.w;
        }
}

// 1 / (1 + e^-x) from the hardware exp2 and reciprocal (one ulp each; e^-x
// overflows to infinity below x = -88, whose reciprocal is the limit, 0).  The
// exponent is rounded once, so the result is off by about 2 |x| 2^-24 of
// itself: 2^-16.5 at the far end, which disappears in a bf16 output.
// EXACT, for fp32 outputs: from e^-|x|, whose exponent's rounding is applied
// to first order, a few 2^-24 everywhere: seven operations more, hidden behind
// HBM at fp32's four values per 16 bytes (16384 x 4096 gated 140 us with and
// without).
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float x)
{
    if constexpr (!EXACT) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
    const float y = fmaxf(-fabsf(x), -256.0f), t = y * 1.44269502f;
    const float r = fmaf(y, 1.44269502f, -t) + y * 1.92596303e-8f;
    float e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e, r * 0.693147182f, e);
    const float q = __builtin_amdgcn_rcpf(1.0f + e);
    return x < 0.0f ? e * q : q;
}

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| <= 1.  The exponent of e
// is rounded once and the rest of the product applied to first order; then
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3, by its series to s^15 (the
// next term is below 2^-28 of the sum).  Relative error a few 2^-24.  e is
// zero in fp32 long before |x| = 256; the bound keeps t and r finite at the
// type's ends.
__device__ __forceinline__ float softplus(float x)
{
    const float y = fmaxf(-fabsf(x), -256.0f), t = y * 1.44269502f;
    const float r = fmaf(y, 1.44269502f, -t) + y * 1.92596303e-8f;
    float e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e, r * 0.693147182f, e);
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e), q = s * s;
    float p = fmaf(q, 1.0f / 15.0f, 1.0f / 13.0f);
    p = fmaf(q, p, 1.0f / 11.0f);
    p = fmaf(q, p, 1.0f / 9.0f);
    p = fmaf(q, p, 1.0f / 7.0f);
    p = fmaf(q, p, 1.0f / 5.0f);
    p = fmaf(q, p, 1.0f / 3.0f);
    return fmaxf(x, 0.0f) + fmaf(2.0f * s * q, p, 2.0f * s);
}

// Sum over aligned groups of N = 16, 32 or 64 lanes, in every lane.
template <int N>
__device__ __forceinline__ float lanes_sum(float x)
{
    x += dpp<DPP_XOR1>(x);
    x += dpp<DPP_XOR2>(x);
    x += dpp<DPP_HALF_MIRROR>(x);
    x += dpp<DPP_MIRROR>(x);
    if constexpr (N >= 32) {
        float a = x, b = x;
        swap16(a, b);
        x = a + b;
    }
    if constexpr (N == 64) {
        float a = x, b = x;
        swap32(a, b);
        x = a + b;
    }
    return x;
}

// Packed sequences.  Sequence b with first row cu[b] owns the tile numbers
// from (cu[b] >> shift) + b up to the next sequence's: at least
// ceil(length / 2^shift) of them, so numbers 0 .. (T >> shift) + n - 1 cover
// every tile without a table, and a number past its sequence's last tile has
// no rows.  seq_of_tile finds the sequence with one probe per lane, 64
// sequences a round (every lane of the wave must take part); with bounds that
// break the rules it still returns a sequence in [0, n).
__device__ __forceinline__ int seq_of_tile(const int32_t *cu, int n, int id, int shift)
{
    const int lane = (int)(__builtin_amdgcn_workitem_id_x() & 63u);
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const long long p = lo + (long long)lane * step;
        bool in = lane == 0;
        if (p < hi && lane) in = (long long)(cu[p] >> shift) + p <= id;
        const int k = __popcll(__ballot(in));
        lo += (k - 1) * step;
        if (lo + step < hi) hi = lo + step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

struct SeqTile {
    int seq;
    int start, len;   // the sequence's first row and its length
    int k;            // the tile's number inside the sequence
    int slot;
};

// The sequence's rows and slot; false when it is empty or skipped.
__device__ __forceinline__ bool seq_rows(const int32_t *cu, const int32_t *slots, int b, int T, int n_slots,
                                         SeqTile &x)
{
    x.seq = b;
    x.start = cu[b];
    const int end = cu[b + 1];
    x.slot = slots ? slots[b] : b;
    if (x.start < 0 || end <= x.start || end > T || x.slot < 0 || x.slot >= n_slots) return false;
    x.len = end - x.start;
    return true;
}

__device__ __forceinline__ bool seq_tile(const int32_t *cu, const int32_t *slots, int n, int id, int shift, int T,
                                         int n_slots, SeqTile &x)
{
    const int b = seq_of_tile(cu, n, id, shift);
    if (!seq_rows(cu, slots, b, T, n_slots, x)) return false;
    x.k = id - ((x.start >> shift) + b);
    return x.k >= 0 && ((long long)x.k << shift) < x.len;
}

}  // namespace gdnq

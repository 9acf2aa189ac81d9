// rotate.hpp -- rotary positions of one head's values (device helpers of
// gdnq_rope and gdnq_kv_append).
//
// The angle of a pair at a position is the product of the position and the
// pair's frequency in units of 2^-64 turns, modulo 2^64: exact in integers,
// whatever the position.
#pragma once

#include <hip/hip_runtime.h>

#include "rows.hpp"

namespace gdnq {

// (cos, sin) of phase 2^-64 turns, times amp.  The phase is rounded to 2^-32
// turns (an error of 2^-30 radians), split into the nearest quarter turn and a
// rest of at most an eighth, |y| <= pi/4, whose series end at y^9 and y^10 (the
// next terms are below 2^-28).
__device__ __forceinline__ float2 turn(unsigned long long phase, float amp)
{
    const unsigned u = (unsigned)((phase + 0x80000000ull) >> 32);
    const unsigned quarter = (u + 0x20000000u) >> 30;
    const float y = (float)(int)(u - (quarter << 30)) * 1.46291807927e-9f;   // 2 pi / 2^32
    const float q = y * y;
    float s = fmaf(q, 2.75573192e-6f, -1.98412698e-4f);
    s = fmaf(q, s, 8.33333333e-3f);
    s = fmaf(q, s, -0.166666667f);
    s = fmaf(y * q, s, y);
    float c = fmaf(q, -2.75573192e-7f, 2.48015873e-5f);
    c = fmaf(q, c, -1.38888889e-3f);
    c = fmaf(q, c, 4.16666667e-2f);
    c = fmaf(q, c, -0.5f);
    c = fmaf(q, c, 1.0f);
    const bool swap = quarter & 1;
    const float a = swap ? s : c, b = swap ? c : s;
    // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
    return make_float2(((quarter + 1) & 2) ? -a * amp : a * amp, (quarter & 2) ? -b * amp : b * amp);
}

// 16 bytes of a row, at any element (the card reads and writes them wherever they
// lie); STREAM: not used again soon, past the caches.
template <bool BF16, bool STREAM>
struct Row16 {
    static constexpr int V = BF16 ? 8 : 4;
    using elem = std::conditional_t<BF16, uint16_t, float>;
    typedef uint32_t words __attribute__((ext_vector_type(4)));
    typedef words anywhere __attribute__((aligned(2)));

    __device__ __forceinline__ static uint4 load(const void *base, size_t off)
    {
        const auto p = reinterpret_cast<const anywhere *>(reinterpret_cast<const elem *>(base) + off);
        if constexpr (STREAM) return __builtin_bit_cast(uint4, (words)__builtin_nontemporal_load(p));
        else return __builtin_bit_cast(uint4, (words)*p);
    }

    __device__ __forceinline__ static void store(void *base, size_t off, const uint4 &r)
    {
        const auto p = reinterpret_cast<anywhere *>(reinterpret_cast<elem *>(base) + off);
        if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(words, r), p);
        else *p = __builtin_bit_cast(words, r);
    }
};

// How a head of d values splits into pieces of one thread: np turn 16 bytes (of
// interleaved pairs, or of each half), nr the pairs that these leave over, one by one, nc
// copy 16 bytes, and the others what is left of the copied values, one by one.
struct HeadPieces {
    int rot, np, nr, nc, ni;
    Divisor byNi;
};

inline HeadPieces head_pieces(int d, int rot, bool inter, bool bf16)
{
    const int v = bf16 ? 8 : 4, turned = inter ? rot : rot / 2;
    HeadPieces p{rot, turned / v, inter ? turned % v / 2 : turned % v, (d - rot) / v, 0, {}};
    p.ni = p.np + p.nr + p.nc + (d - rot) % v;
    p.byNi = make_divisor((unsigned)p.ni);
    return p;
}

__device__ __forceinline__ void turn_pair(float &a, float &b, const float2 &t)
{
    const float u = a, w = b;
    a = fmaf(u, t.x, -w * t.y);
    b = fmaf(w, t.x, u * t.y);
}

// Piece `it` of a head at element xo of x into the head at element yo of y;
// cs: the row's (cos, sin) pairs.
template <bool BF16, bool INTER, bool STREAM>
__device__ __forceinline__ void turn_piece(const void *x, size_t xo, void *y, size_t yo, int it, const float2 *cs,
                                           const HeadPieces &p)
{
    using R = Row16<BF16, STREAM>;
    constexpr int V = R::V;
    using P = Pack<BF16, V>;
    if (it < p.np) {
        if constexpr (INTER) {
            float v[V];
            P::widen(R::load(x, xo + it * V), v);
#pragma unroll
            for (int i = 0; i < V / 2; i++) turn_pair(v[2 * i], v[2 * i + 1], cs[it * (V / 2) + i]);
            R::store(y, yo + it * V, P::narrow(v));
        } else {
            const int ja = it * V, jb = p.rot / 2 + it * V;
            float a[V], b[V];
            const uint4 ra = R::load(x, xo + ja), rb = R::load(x, xo + jb);
            P::widen(ra, a);
            P::widen(rb, b);
#pragma unroll
            for (int i = 0; i < V; i++) turn_pair(a[i], b[i], cs[ja + i]);
            R::store(y, yo + ja, P::narrow(a));
            R::store(y, yo + jb, P::narrow(b));
        }
        return;
    }
    it -= p.np;
    if (it < p.nr) {
        const int pair = p.np * (INTER ? V / 2 : V) + it;
        const int ja = INTER ? 2 * pair : pair, jb = INTER ? ja + 1 : p.rot / 2 + pair;
        float a = load1<BF16>(x, xo + ja), b = load1<BF16>(x, xo + jb);
        turn_pair(a, b, cs[pair]);
        store1<BF16>(y, yo + ja, a);
        store1<BF16>(y, yo + jb, b);
        return;
    }
    it -= p.nr;
    if (it < p.nc) {
        const int j = p.rot + it * V;
        R::store(y, yo + j, R::load(x, xo + j));
    } else {   // as it is, without arithmetic
        using elem = typename R::elem;
        const int j = p.rot + p.nc * V + it - p.nc;
        reinterpret_cast<elem *>(y)[yo + j] = reinterpret_cast<const elem *>(x)[xo + j];
    }
}

// Whether a call's rows, read and written, are more than the caches would keep.
inline bool streams(unsigned long long bytes) { return bytes >= 64ull << 20; }

}  // namespace gdnq

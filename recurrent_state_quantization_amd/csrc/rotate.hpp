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

// How a head of d values splits into pieces of one thread: np that turn (V
// pairs, or V values of interleaved pairs), then the copied ones of V values.
struct HeadPieces {
    int rot, np, ni;
    Divisor byNi;
};

// Whether heads of d values (their rows in 16-byte pieces) split into pieces of 16 bytes.
inline bool wide_pieces(int d, int rot, bool inter, int es)
{
    const int v = 16 / es;
    return d % v == 0 && (d - rot) % v == 0 && (inter ? rot : rot / 2) % v == 0;
}

inline HeadPieces head_pieces(int d, int rot, bool inter, int v)
{
    HeadPieces p{rot, 0, 0, {}};
    p.np = inter && v > 1 ? rot / v : rot / 2 / v;
    p.ni = p.np + (d - rot) / v;
    p.byNi = make_divisor((unsigned)p.ni);
    return p;
}

// Piece `it` of a head at element xo of x into the head at element yo of y;
// cs: the row's (cos, sin) pairs.
template <bool BF16, int V, bool INTER, bool STREAM>
__device__ __forceinline__ void turn_piece(const void *x, size_t xo, void *y, size_t yo, int it, const float2 *cs,
                                           const HeadPieces &p)
{
    using P = Pack<BF16, V>;
    if (it >= p.np) {
        const int j = p.rot + (it - p.np) * V;
        P::template store_once<STREAM>(y, yo + j, P::template load_once<STREAM>(x, xo + j));
    } else if constexpr (INTER && V > 1) {
        float v[V];
        P::widen(P::template load_once<STREAM>(x, xo + it * V), v);
#pragma unroll
        for (int i = 0; i < V / 2; i++) {
            const float2 t = cs[it * (V / 2) + i];
            const float a = v[2 * i], b = v[2 * i + 1];
            v[2 * i] = fmaf(a, t.x, -b * t.y);
            v[2 * i + 1] = fmaf(b, t.x, a * t.y);
        }
        P::template store_once<STREAM>(y, yo + it * V, P::narrow(v));
    } else {
        const int ja = INTER ? 2 * it : it * V, jb = INTER ? 2 * it + 1 : p.rot / 2 + it * V;
        float a[V], b[V];
        const typename P::raw ra = P::template load_once<STREAM>(x, xo + ja);
        const typename P::raw rb = P::template load_once<STREAM>(x, xo + jb);
        P::widen(ra, a);
        P::widen(rb, b);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float2 t = cs[it * V + i];
            const float u = a[i], w = b[i];
            a[i] = fmaf(u, t.x, -w * t.y);
            b[i] = fmaf(w, t.x, u * t.y);
        }
        P::template store_once<STREAM>(y, yo + ja, P::narrow(a));
        P::template store_once<STREAM>(y, yo + jb, P::narrow(b));
    }
}

// Whether a call's rows, read and written, are more than the caches would keep.
inline bool streams(unsigned long long bytes) { return bytes >= 64ull << 20; }

}  // namespace gdnq

// layer_launchers.hpp -- prototypes of the launchers behind
// include/gdnq_layer.h (internal).  Arguments are validated by
// layer_api.cpp, which also fills in the row distances.
#pragma once

#include <hip/hip_runtime.h>

#include "gdnq_layer.h"
#include "launch.hpp"

namespace gdnq {

struct ConvCall {
    const void *x;
    const float *w, *bias;
    void *state, *y;
    const int32_t *slots, *cont, *cu;
    long long ldx, ldy;
    int n_slots, n, T;
};

// Calls of this many token rows or fewer leave every sequence of the scan whole.
constexpr int SSM_WHOLE = 384;

struct SsmCall {
    gdnq_ssm_io io;   // row distances filled in
    float *S;
    const int32_t *slots, *cont, *cu;
    int n_slots, n, T;
    void *ws;
};

struct NormCall {
    const void *x, *z, *res;
    void *y, *res_out;
    const float *w, *post_w;
    long long ldx, ldz, ldr, ldro, ldy;
    float scale;
    int rows;
};

hipError_t launch_conv_prefill(const gdnq_conv_desc &d, const ConvCall &c, hipStream_t st);
hipError_t launch_conv_step(const gdnq_conv_desc &d, const ConvCall &c, hipStream_t st);
hipError_t launch_ssm_step(const gdnq_ssm_desc &d, const SsmCall &c, hipStream_t st);
size_t ssm_workspace(const gdnq_ssm_desc &d, int n, int T);
hipError_t launch_ssm_prefill(const gdnq_ssm_desc &d, const SsmCall &c, hipStream_t st);
hipError_t launch_norm_gated(const gdnq_norm_desc &d, const NormCall &c, hipStream_t st);
hipError_t launch_norm_residual(const gdnq_norm_desc &d, const NormCall &c, hipStream_t st);

// The grid of `blocks` workgroups or a few more.  One dimension holds fewer than
// 2^32 threads, which narrow rows and small groups pass at a few GB: such calls
// take two, whose workgroups block_id() numbers through.
inline dim3 grid_of(unsigned long long blocks, unsigned threads)
{
    const unsigned long long most = 0xFFFFFFFFull / threads, ny = (blocks + most - 1) / most;
    return dim3((unsigned)((blocks + ny - 1) / ny), (unsigned)ny);
}

// Whether rows at p, ld elements of `es` bytes apart, can be read in 16-byte
// pieces.
inline bool wide_rows(const void *p, long long ld, int es)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0;
}

}  // namespace gdnq

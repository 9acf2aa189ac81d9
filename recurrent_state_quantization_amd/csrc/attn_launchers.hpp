// attn_launchers.hpp -- prototypes of the launchers behind
// include/gdnq_attn.h (internal).  Arguments are validated by attn_api.cpp,
// which also fills in the defaults of descriptors and distances.
#pragma once

#include <hip/hip_runtime.h>

#include "gdnq_attn.h"
#include "launch.hpp"
#include "layer_launchers.hpp"

namespace gdnq {

struct RopeCall {
    const void *x;
    void *y;
    const uint64_t *table;
    const int32_t *pos;
    long long ldx, ldy;
    int H, rows;
};

struct AppendCall {
    gdnq_kv kv;
    const void *q, *k, *v;
    void *q_out;
    const uint64_t *table;
    const int32_t *pos, *slots, *cu;
    long long ldq, ldqo, ldk, ldv;
    int n, T;
};

struct AttnCall {
    gdnq_kv kv;
    const void *q;
    void *o;
    const int32_t *slots;
    long long ldq, ldo;
    int n;
    void *ws;
};

struct EvictCall {
    gdnq_kv kv;
    const int32_t *slots;
    int budget, sink, recent, n;
    void *ws;
};

hipError_t launch_rope(const gdnq_rope_desc &d, const RopeCall &c, hipStream_t st);
// whether 31 bits number the pieces of a workgroup's rows
bool kv_append_numbers(const gdnq_attn_desc &d, const gdnq_rope_desc *r, const AppendCall &c);
hipError_t launch_kv_append(const gdnq_attn_desc &d, const gdnq_rope_desc *r, const AppendCall &c, hipStream_t st);
size_t attn_workspace(const gdnq_attn_desc &d, const gdnq_kv &kv, int n);
hipError_t launch_attn_step(const gdnq_attn_desc &d, const AttnCall &c, hipStream_t st);
size_t kv_evict_workspace(const gdnq_attn_desc &d, const gdnq_kv &kv, int budget, int n);
hipError_t launch_kv_evict(const gdnq_attn_desc &d, const EvictCall &c, hipStream_t st);

}  // namespace gdnq

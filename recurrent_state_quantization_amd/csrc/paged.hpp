// paged.hpp -- the paged cache of keys and values on the device (helpers of
// the kernels behind include/gdnq_attn.h).
#pragma once

#include <hip/hip_runtime.h>

#include "gdnq_attn.h"

namespace gdnq {

// A slot's rows: its table, and how many it holds.
struct SlotRows {
    const int32_t *table;
    int len;
};

// Entry i's slot; false: the entry is skipped.
__device__ __forceinline__ bool slot_rows(const gdnq_kv &kv, const int32_t *slots, int i, int shift, SlotRows &x)
{
    const int slot = slots ? slots[i] : i;
    if (slot < 0 || slot >= kv.n_slots) return false;
    x.len = kv.lens[slot];
    x.table = kv.table + (size_t)slot * kv.max_pages;
    return x.len >= 0 && x.len <= (kv.max_pages << shift);
}

// Element of row `off` of page p and head h in k and v, and in acc and pos.
__device__ __forceinline__ size_t row_at(const gdnq_kv &kv, int p, int h, int off)
{
    return (size_t)p * kv.ldp + (size_t)h * kv.ldh + (size_t)off * kv.ldr;
}

__device__ __forceinline__ size_t sum_at(int hk, int shift, int p, int h, int off)
{
    return (((size_t)p * hk + h) << shift) + off;
}

}  // namespace gdnq

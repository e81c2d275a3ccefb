// attend.h - internal launchers of the operators of kvattend.h (host side),
// and the layout of a paged cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layout.h"

namespace kvc {

// bf16 head vectors: element (n, h, c) at data[n * ts + h * hs + c].
struct RowsDev {
    uint16_t* data;
    uint64_t ts, hs;
};

// Byte layout of one page (see kvattend.h): codes, then (8-bit formats) steps.
struct PageLayout {
    uint32_t num_pages, H, P, d, format;
    uint32_t esize;        // bytes of one code
    uint64_t steps;        // offset of the steps in a page
    uint64_t page_bytes;
};

inline bool page_spec_ok(uint32_t num_pages, uint32_t H, uint32_t P, uint32_t d, uint32_t format) {
    return num_pages >= 1 && num_pages <= 0x7FFFFFFFu && H >= 1 && H <= (1u << 16) &&
           (P == 16 || P == 32 || P == 64 || P == 128 || P == 256) && (d == 64 || d == 128) && format <= 2;
}

inline PageLayout page_layout(uint32_t num_pages, uint32_t H, uint32_t P, uint32_t d, uint32_t format) {
    PageLayout l;
    l.num_pages = num_pages;
    l.H = H;
    l.P = P;
    l.d = d;
    l.format = format;
    l.esize = format == 0 ? 2 : 1;
    l.steps = 2ull * H * P * d * l.esize;
    l.page_bytes = align_up(l.steps + (format == 0 ? 0 : 2ull * H * P * 4), 256);
    return l;
}

constexpr int kMaxPairs = 64;
struct RotateArgs {
    uint32_t n, Hq, Hk, d;
    RowsDev q_in, k_in, q_out, k_out;
    const void *q_weight, *k_weight;
    float eps;
    const int64_t* positions;
    const float* inv_freq;  // host
    uint32_t n_pairs, pairing;
};
hipError_t launch_norm_rotate(const RotateArgs& a, hipStream_t stream);

hipError_t launch_page_write(const PageLayout& l, void* pages, uint32_t n, const RowsDev& k, const RowsDev& v,
                             const int64_t* slots, int32_t* dev_status, hipStream_t stream);
hipError_t launch_page_read(const PageLayout& l, const void* pages, uint32_t n, const int64_t* slots,
                            const RowsDev& k_out, const RowsDev& v_out, int32_t* dev_status, hipStream_t stream);

// How the tokens of one source (a pool's layer, or pages) are shared out among
// workgroups. A unit is the work of one kv head of one sequence (of all
// agents for a pool) for 16 rt query rows.
struct AttendPlan {
    uint32_t rows;        // query rows that share a kv head's tokens
    uint32_t rt;          // row tiles of 16 of one wave: 1 or 2
    uint32_t row_blocks;  // units that share tokens, ceil(rows / (16 rt))
    bool whole;           // each workgroup takes one unit
    uint64_t units, W;    // W: workgroups
    uint64_t blocks;      // blocks of tokens of all units, at most
    uint64_t slots;       // places for partial results: 16 rt rows of d sums, a maximum and a sum
    // Bytes that serve this plan and that of every call with fewer sequences, rows or
    // tokens: never less for more of them, where `bytes` falls (a call whose units are
    // whole needs no places at all).
    uint64_t room;
    uint64_t part_bytes(uint32_t d) const { return slots * 16 * rt * (d + 2) * 4; }
    uint64_t bytes_of(uint64_t places, uint32_t d) const { return align_up(places * 16 * rt * (d + 2) * 4 + units * 8, 256); }
    uint64_t bytes(uint32_t d) const { return bytes_of(slots, d); }
};
// tail: pages behind a pool (all parts are joined, none is written as output).
AttendPlan page_attend_plan(uint32_t n_seqs, uint32_t H, uint32_t Hq, uint32_t d, uint64_t max_tokens, bool tail);
AttendPlan pool_attend_plan(uint32_t H, uint32_t n_agents, uint32_t Hq, uint32_t d, uint32_t T, bool tail);

struct TailArgs {
    PageLayout lay;
    const uint8_t* pages;
    const int32_t* table;
    uint32_t table_cols;
    uint64_t table_stride;
    const int32_t* lens;
};
struct AttendArgs {
    uint32_t n, H, Hq, d;  // sequences (agents), kv heads, query heads, channels
    RowsDev q, out;
    float scale;
    float* lse;
    void* ws;
    int32_t* status;
    // pool (pool != nullptr)
    const uint8_t* pool;
    uint32_t L, T, layer;
    // pages (table != nullptr)
    TailArgs tail;
};
hipError_t launch_attend(const AttendArgs& a, hipStream_t stream);

#ifdef __HIPCC__
// Asks for every 64-byte line of the kernel's arguments (BYTES of them) at
// once: read where they are first used, each line costs a latency of its own
// (attention over one short sequence 6.0 -> 5.6 us, its join 4.1 -> 3.9).
template <int BYTES>
__device__ __forceinline__ void fetch_arguments() {
    const auto* a = (const __attribute__((address_space(4))) uint32_t*)__builtin_amdgcn_kernarg_segment_ptr();
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < BYTES / 4; i += 16) all |= a[i];
    asm volatile("" ::"s"(all));
}
#endif

}  // namespace kvc

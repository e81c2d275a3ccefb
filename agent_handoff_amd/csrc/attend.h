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

// KVC_PAGE_*
constexpr int kPageBf16 = 0, kPageInt8 = 1, kPageFp8 = 2, kPageFp4 = 4;
constexpr uint32_t kFp4Block = 32;  // channels that share a power of two

// Byte layout of one page (see kvattend.h): codes, then (but for bf16) steps.
struct PageLayout {
    uint32_t num_pages, H, P, d, format;
    uint64_t steps;        // offset of the steps in a page
    uint64_t page_bytes;
};

// Bytes of a vector's codes, and of its step or steps.
KVC_HD constexpr uint32_t page_code_bytes(int format, uint32_t d) {
    return format == kPageBf16 ? 2 * d : format == kPageFp4 ? d / 2 : d;
}
KVC_HD constexpr uint32_t page_step_bytes(int format, uint32_t d) {
    return format == kPageBf16 ? 0 : format == kPageFp4 ? d / kFp4Block : 4;
}

inline bool page_spec_ok(uint32_t num_pages, uint32_t H, uint32_t P, uint32_t d, uint32_t format) {
    return num_pages >= 1 && num_pages <= 0x7FFFFFFFu && H >= 1 && H <= (1u << 16) &&
           (P == 16 || P == 32 || P == 64 || P == 128 || P == 256) && (d == 64 || d == 128) &&
           (format <= 2 || format == kPageFp4);
}

inline PageLayout page_layout(uint32_t num_pages, uint32_t H, uint32_t P, uint32_t d, uint32_t format) {
    PageLayout l;
    l.num_pages = num_pages;
    l.H = H;
    l.P = P;
    l.d = d;
    l.format = format;
    l.steps = 2ull * H * P * page_code_bytes(format, d);
    l.page_bytes = align_up(l.steps + 2ull * H * P * page_step_bytes(format, d), 256);
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

// Norms, rotation and the write (kvpage_append).
struct AppendArgs {
    uint32_t n, Hq;
    PageLayout lay;
    uint8_t* pages;
    RowsDev q_in, k_in, v_in, q_out;
    const void *q_weight, *k_weight;
    float eps;
    const int64_t* positions;
    const float* inv_freq;  // host
    uint32_t n_pairs, pairing;
    const int64_t* slots;
    int32_t* status;
};
hipError_t launch_append(const AppendArgs& a, hipStream_t stream);

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
// Many new tokens, few of each sequence.
AttendPlan many_attend_plan(uint32_t n_seqs, uint32_t n_tokens, uint32_t H, uint32_t Hq, uint32_t d, uint64_t max_tokens,
                            uint32_t window, uint32_t sinks);
// Workspace of any such call with up to `rows` query rows of all sequences and a kv head.
uint64_t many_attend_room(uint32_t n_seqs, uint64_t rows, uint32_t H, uint32_t d, uint64_t max_tokens);
AttendPlan pool_attend_plan(uint32_t H, uint32_t n_agents, uint32_t Hq, uint32_t d, uint32_t T, bool tail);

// Tokens that a call over at most max_tokens counts for a sequence, at most: with a
// window, its tokens and the sinks, each up to the next run of 16.
inline uint64_t seen_tokens(uint64_t max_tokens, uint64_t window, uint64_t sinks) {
    if (!window) return max_tokens;
    const uint64_t most = window + align_up(sinks, 16) + 15;
    return most < max_tokens ? most : max_tokens;
}

struct TailArgs {
    PageLayout lay;
    const uint8_t* pages;
    const int32_t* table;
    uint32_t table_cols;
    uint64_t table_stride;
    const int32_t* lens;
    uint32_t window, sinks;  // window 0: every token
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
    // many new tokens of each sequence, over pages alone (starts != nullptr)
    const int32_t* starts;
    uint32_t tokens;
};
hipError_t launch_attend(const AttendArgs& a, hipStream_t stream);

// Attention of many new tokens. The query rows of a sequence and kv head (tokens x
// the heads that share it) are taken in blocks; `blocks` bounds how many a kv head
// has, which the host does not know.
constexpr uint32_t kPromptRows = 64;  // a call's limit counts blocks of so many rows
struct PromptPlan {
    bool few;         // few new tokens of each sequence: taken by launch_attend
    uint32_t shares;  // workgroups that share out a kv head's tiles evenly (0: each takes a block)
    uint64_t blocks;  // of a kv head, at most
    uint64_t bytes;   // of the workspace: what the call uses,
    uint64_t room;    // and what serves every smaller call too
};
PromptPlan prompt_plan(uint32_t n_seqs, uint32_t n_tokens, uint32_t H, uint32_t Hq, uint32_t d, uint64_t max_tokens,
                       uint32_t window, uint32_t sinks);
struct PromptArgs {
    uint32_t n, rows, H, Hq, d;  // sequences, query rows (tokens), kv heads, query heads, channels
    RowsDev q, out;
    float scale;
    float* lse;
    void* ws;
    int32_t* status;
    const int32_t* starts;
    TailArgs tail;
};
hipError_t launch_attend_prompt(const PromptArgs& a, const PromptPlan& plan, hipStream_t stream);

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

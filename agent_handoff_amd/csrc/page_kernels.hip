// page_kernels.hip - the paged cache: quantising tokens as they are written,
// and reading them back, for gfx950.
//
// d / 8 lanes take one head vector, 8 channels (one 16-byte chunk) each, so
// every access of bf16 rows and of codes is one contiguous run per vector. (Four
// lanes share the power of two of 4-bit codes.)
// Both directions are bound by memory alone: 2 d bytes on one side, d + 4
// (bf16: 2 d, 4 bits: d / 2 + d / 32) on the other. 32768 tokens of 8 heads of 128 read back from int8
// pages: 34.3 us, 5.9 TB/s; 8191 tokens written to e4m3 slots in random order:
// 11.9 us, 4.3 TB/s (the 4-byte steps of scattered slots each move a line). 4 bits, 8191 tokens
// of 8 heads of 128 laid out by heads: 9.5 us to write, 10.4 to read back (42 MB: 4.4 and 4.0 TB/s).
#include "page_codes.h"

namespace kvc {
namespace {

constexpr int kDevBadSlot = 16;  // KVC_DEV_BAD_SLOT

struct PageParams {
    uint8_t* pages;
    RowsDev rows[2];  // keys, values
    const int64_t* slots;
    int32_t* status;
    uint32_t n, H, P, num_pages;
    uint64_t steps, page_bytes;
    uint32_t heads_inner;  // tokens hold their heads next to one another
    uint32_t vecs;         // of one row of the grid: n * H, or n of one head
};

// One vector: whether there is one, its token's slot (as given), the element
// offset of its row and the line it takes in a page but for the slot's.
struct Vector {
    bool live;
    int64_t slot;
    uint64_t row;
    uint64_t line;
};

// Vector `at` of this workgroup's row of the grid: keys or values (z); with
// heads inside tokens, (token, head) = at / H, else token `at` of head y. Its slot
// is on its way; nothing waits for it here.
__device__ __forceinline__ Vector vector_of(const PageParams& p, uint32_t at) {
    Vector x;
    x.live = at < p.vecs;
    at = x.live ? at : p.vecs - 1;
    const uint32_t kv = blockIdx.z;
    const uint32_t tok = p.heads_inner ? at / p.H : at, h = p.heads_inner ? at - tok * p.H : blockIdx.y;
    x.slot = p.slots[tok];
    x.row = tok * p.rows[kv].ts + h * p.rows[kv].hs;
    x.line = ((uint64_t)kv * p.H + h) * p.P;
    return x;
}

// Its byte offsets in the cache: of its codes and its step (or steps). A vector whose slot
// is outside the cache, or negative, is not live, and has those of slot 0.
struct Place {
    uint64_t code, step;
};
template <int FMT, int D>
__device__ __forceinline__ Place place_of(const PageParams& p, Vector& x) {
    const bool inside = x.slot >= 0 && (uint64_t)x.slot < (uint64_t)p.num_pages * p.P;
    x.live = x.live && inside;
    const uint64_t s = inside ? (uint64_t)x.slot : 0;
    const uint32_t shift = 31 - __clz(p.P);
    const uint64_t page = s >> shift, line = x.line + (s & (p.P - 1));
    return Place{page * p.page_bytes + line * page_code_bytes(FMT, D),
                 page * p.page_bytes + p.steps + line * page_step_bytes(FMT, D)};
}
__device__ __forceinline__ void report(const PageParams& p, int64_t slot) {
    if (slot >= 0 && (uint64_t)slot >= (uint64_t)p.num_pages * p.P && p.status) atomicOr(p.status, kDevBadSlot);
}

// U vectors of each group of lanes at a time: their slots and rows are asked for
// together, before any is waited for (8191 tokens written: 11.1 us;
// one after another, 13.5).
template <int FMT, int D, int U>
__global__ __launch_bounds__(kBlockThreads) void page_write_kernel(PageParams p) {
    constexpr int LPV = D / 8;
    constexpr uint32_t VPB = kBlockThreads / LPV;
    const uint32_t i = threadIdx.x % LPV;
    const uint32_t v0 = blockIdx.x * (VPB * U) + threadIdx.x / LPV;
    Vector vec[U];
    kvc_u32x4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        vec[u] = vector_of(p, v0 + u * VPB);
        x[u] = *reinterpret_cast<const kvc_u32x4*>(p.rows[blockIdx.z].data + vec[u].row + 8 * i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Place at = place_of<FMT, D>(p, vec[u]);
        const uint4 y = make_uint4(x[u].x, x[u].y, x[u].z, x[u].w);
        if (FMT == kPageBf16) {
            if (vec[u].live) *reinterpret_cast<kvc_u32x4*>(p.pages + at.code + 16 * i) = x[u];
        } else if (FMT == kPageFp4) {
            uint32_t power;
            const uint32_t c = quantise8_fp4(y, max_lanes<kFp4Block / 8>(magnitude8(y)), power);
            if (vec[u].live) {
                *reinterpret_cast<uint32_t*>(p.pages + at.code + 4 * i) = c;
                if (i % 4 == 0) p.pages[at.step + i / 4] = (uint8_t)power;
            }
        } else {
            float step;
            const uint2 c = quantise8<FMT>(y, max_lanes<LPV>(magnitude8(y)), step);
            if (vec[u].live) {
                *reinterpret_cast<uint2*>(p.pages + at.code + 8 * i) = c;
                if (i == 0) *reinterpret_cast<float*>(p.pages + at.step) = step;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) report(p, vec[u].slot);
}

template <int FMT, int D, int U>
__global__ __launch_bounds__(kBlockThreads) void page_read_kernel(PageParams p) {
    constexpr int LPV = D / 8;
    constexpr uint32_t VPB = kBlockThreads / LPV;
    const uint32_t i = threadIdx.x % LPV;
    const uint32_t v0 = blockIdx.x * (VPB * U) + threadIdx.x / LPV;
    Vector vec[U];
    uint4 x[U];
    uint2 c[U];
    float step[U];
#pragma unroll
    for (int u = 0; u < U; ++u) vec[u] = vector_of(p, v0 + u * VPB);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Place at = place_of<FMT, D>(p, vec[u]);
        if (FMT == kPageBf16) {
            x[u] = *reinterpret_cast<const uint4*>(p.pages + at.code + 16 * i);
        } else if (FMT == kPageFp4) {
            c[u].x = *reinterpret_cast<const uint32_t*>(p.pages + at.code + 4 * i);
            c[u].y = p.pages[at.step + i / 4];
        } else {
            c[u] = *reinterpret_cast<const uint2*>(p.pages + at.code + 8 * i);
            step[u] = *reinterpret_cast<const float*>(p.pages + at.step);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (FMT == kPageFp4)
            x[u] = dequantise8_fp4(c[u].x, c[u].y);
        else if (FMT != kPageBf16)
            x[u] = dequantise8<FMT>(c[u], step[u]);
        if (vec[u].live) st_stream(reinterpret_cast<uint4*>(p.rows[blockIdx.z].data + vec[u].row + 8 * i), x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) report(p, vec[u].slot);
}

PageParams page_params(const PageLayout& l, const void* pages, uint32_t n, const RowsDev& k, const RowsDev& v,
                       const int64_t* slots, int32_t* dev_status) {
    PageParams p{};
    p.pages = static_cast<uint8_t*>(const_cast<void*>(pages));
    p.rows[0] = k;
    p.rows[1] = v;
    p.slots = slots;
    p.status = dev_status;
    p.n = n;
    p.H = l.H;
    p.P = l.P;
    p.num_pages = l.num_pages;
    p.steps = l.steps;
    p.page_bytes = l.page_bytes;
    // follow the rows' order in memory; a launch has fewer than 2^32 threads, 4 for a vector here
    p.heads_inner = k.hs <= k.ts && (uint64_t)n * l.H < (1u << 29);
    p.vecs = p.heads_inner ? n * l.H : n;
    return p;
}

// Four vectors for each group of lanes where that still fills the GPU: 8 heads of 128, us with one and with four,
// 2048 tokens bf16 written 3.8 and 4.0, read 3.2 and 3.4, e4m3 4.3 and 5.0, 3.4 and 3.7; 4096 (from where it is
// taken) 5.7 and 5.4, 4.5 and 4.3, e4m3 6.5 and 7.0, 4.5 and 4.6; 8192 11.8 and 11.0, 8.8 and 9.2, e4m3 11.6 and
// 11.3, 7.6 and 7.2.
template <int FMT, int D>
hipError_t launch_page(bool write, const PageParams& p, hipStream_t stream) {
    constexpr uint32_t VPB = kBlockThreads / (D / 8);
    const bool many = 2ull * p.n * p.H >= 4ull * VPB * 1024;
    const uint32_t per = many ? 4 * VPB : VPB;
    const dim3 grid((p.vecs + per - 1) / per, p.heads_inner ? 1 : p.H, 2), block(kBlockThreads);
    if (write)
        return launch_kernel(many ? page_write_kernel<FMT, D, 4> : page_write_kernel<FMT, D, 1>, grid, block, stream, p);
    return launch_kernel(many ? page_read_kernel<FMT, D, 4> : page_read_kernel<FMT, D, 1>, grid, block, stream, p);
}

template <int D>
hipError_t launch_page_of(bool write, uint32_t format, const PageParams& p, hipStream_t stream) {
    switch (format) {
        case kPageBf16: return launch_page<kPageBf16, D>(write, p, stream);
        case kPageInt8: return launch_page<kPageInt8, D>(write, p, stream);
        case kPageFp8: return launch_page<kPageFp8, D>(write, p, stream);
        default: return launch_page<kPageFp4, D>(write, p, stream);
    }
}
hipError_t launch_page_any(bool write, const PageLayout& l, const PageParams& p, hipStream_t stream) {
    return l.d == 64 ? launch_page_of<64>(write, l.format, p, stream) : launch_page_of<128>(write, l.format, p, stream);
}

}  // namespace

hipError_t launch_page_write(const PageLayout& l, void* pages, uint32_t n, const RowsDev& k, const RowsDev& v,
                             const int64_t* slots, int32_t* dev_status, hipStream_t stream) {
    return launch_page_any(true, l, page_params(l, pages, n, k, v, slots, dev_status), stream);
}

hipError_t launch_page_read(const PageLayout& l, const void* pages, uint32_t n, const int64_t* slots,
                            const RowsDev& k_out, const RowsDev& v_out, int32_t* dev_status, hipStream_t stream) {
    return launch_page_any(false, l, page_params(l, pages, n, k_out, v_out, slots, dev_status), stream);
}

}  // namespace kvc

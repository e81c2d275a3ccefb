// page_kernels.hip - the paged cache: quantising tokens as they are written,
// and reading them back, for gfx950.
//
// d / 8 lanes take one head vector, 8 channels (one 16-byte chunk) each, so
// every access of bf16 rows and of codes is one contiguous run per vector.
// Both directions are bound by memory alone: 2 d bytes on one side, d + 4
// (bf16: 2 d) on the other. 32768 tokens of 8 heads of 128 read back from int8
// pages: 34.3 us, 5.9 TB/s; 8191 tokens written to e4m3 slots in random order:
// 11.9 us, 4.3 TB/s (the 4-byte steps of scattered slots each move a line).
#include "attend.h"
#include "kernels_common.h"

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

// Maximum over the LPV (8 or 16) lanes of a vector.
template <int LPV>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
    const auto step = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
    v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad_perm xor 1
    v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // quad_perm xor 2
    v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // row_half_mirror
    if (LPV == 16) v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));  // row_mirror
    return v;
}

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

// Its byte offsets in the cache: of its codes and its step. A vector whose slot
// is outside the cache, or negative, is not live, and has those of slot 0.
struct Place {
    uint64_t code, step;
};
template <int D, int ES>
__device__ __forceinline__ Place place_of(const PageParams& p, Vector& x) {
    const bool inside = x.slot >= 0 && (uint64_t)x.slot < (uint64_t)p.num_pages * p.P;
    x.live = x.live && inside;
    const uint64_t s = inside ? (uint64_t)x.slot : 0;
    const uint32_t shift = 31 - __clz(p.P);
    const uint64_t page = s >> shift, line = x.line + (s & (p.P - 1));
    return Place{page * p.page_bytes + line * (D * ES), page * p.page_bytes + p.steps + line * 4};
}
__device__ __forceinline__ void report(const PageParams& p, int64_t slot) {
    if (slot >= 0 && (uint64_t)slot >= (uint64_t)p.num_pages * p.P && p.status) atomicOr(p.status, kDevBadSlot);
}

__device__ __forceinline__ void unpack8(const uint4& x, float (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = bf16_lo(w[i]);
        y[2 * i + 1] = bf16_hi(w[i]);
    }
}

// 8 channels of a vector -> codes (8 bytes) and the vector's step.
//
// code = round(x * M / m), m the vector's maximum. With m brought to A in
// [1/2, 1) by a power of two, x * (M * that power) is exact in binary32 (8 + 7
// bits), and q = x * M / m by a reciprocal is corrected by its exact remainder: a
// quotient that is a tie (representable) comes out exact; any other is at
// least 2^-13 of its size away from a tie, since it is a ratio of integers of few
// bits. So the codes are those of exact arithmetic. The step m / M is made the
// same way, correctly rounded (so for each of the 128 significands of m).
// Maxima below 2^-100 take the slow way: their factors leave binary32's range.
template <int FMT, int LPV>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float& step) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;  // magnitudes as integers: NaN above Inf above the rest
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
        const uint32_t y = lo > hi ? lo : hi;
        m = y > m ? y : m;
    }
    m = max_lanes<LPV>(m);
    const float most = FMT == 1 ? 127.0f : 448.0f, inv_most = 1.0f / most;
    const float big = __uint_as_float(m << 16);
    float y[8], q[8];
    unpack8(x, y);
    const int e = __builtin_amdgcn_frexp_expf(big);
    const float A = __builtin_amdgcn_ldexpf(big, -e);
    const float rA = __builtin_amdgcn_rcpf(A);
    const auto corrected = [](float r, float divisor, float reciprocal) {
        const float q0 = r * reciprocal;
        return fmaf(fmaf(-q0, divisor, r), reciprocal, q0);
    };
    if (m >= 0x0D80u) {  // 2^-100
        step = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __builtin_amdgcn_ldexpf(corrected(A, most, inv_most), e);
        if (m >= 0x7F80u) return make_uint2(0, 0);
        const float up = __builtin_amdgcn_ldexpf(most, -e);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = corrected(y[i] * up, A, rA);
    } else {
        step = big / most;
        if (m == 0) return make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = corrected(__builtin_amdgcn_ldexpf(y[i], -e) * most, A, rA);
    }
    if (FMT == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = copysignf(q[i], y[i]);  // the remainder of -0 is +0: e4m3 keeps the sign
    }
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (FMT == 1) {
            // adding 1.5 * 2^23 rounds to an integer (ties to even) held in the low bits
            uint32_t b[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) b[u] = __float_as_uint(q[4 * i + u] + 12582912.0f);
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
            o[i] = lo | hi;
        } else {
            int v = 0;
            v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], v, false);
            v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], v, true);
            o[i] = (uint32_t)v;
        }
    }
    return make_uint2(o[0], o[1]);
}

template <int FMT>
__device__ __forceinline__ uint4 dequantise8(const uint2& c, float step) {
    float y[8];
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (FMT == 1) {
#pragma unroll
            for (int u = 0; u < 4; ++u) y[4 * i + u] = (float)(int32_t)(int8_t)(w[i] >> (8 * u) & 0xFF) * step;
        } else {
            y[4 * i] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 0) * step;
            y[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 1) * step;
            y[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 2) * step;
            y[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 3) * step;
        }
    }
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
}

// U vectors of each group of lanes at a time: their slots and rows are asked for
// together, before any is waited for (8191 tokens written: 11.1 us;
// one after another, 13.5).
template <int FMT, int D, int U>
__global__ __launch_bounds__(kBlockThreads) void page_write_kernel(PageParams p) {
    constexpr int LPV = D / 8, ES = FMT == 0 ? 2 : 1;
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
        const Place at = place_of<D, ES>(p, vec[u]);
        if (FMT == 0) {
            if (vec[u].live) *reinterpret_cast<kvc_u32x4*>(p.pages + at.code + 16 * i) = x[u];
        } else {
            float step;
            const uint2 c = quantise8<FMT, LPV>(make_uint4(x[u].x, x[u].y, x[u].z, x[u].w), step);
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
    constexpr int LPV = D / 8, ES = FMT == 0 ? 2 : 1;
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
        const Place at = place_of<D, ES>(p, vec[u]);
        if (FMT == 0) {
            x[u] = *reinterpret_cast<const uint4*>(p.pages + at.code + 16 * i);
        } else {
            c[u] = *reinterpret_cast<const uint2*>(p.pages + at.code + 8 * i);
            step[u] = *reinterpret_cast<const float*>(p.pages + at.step);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (FMT != 0) x[u] = dequantise8<FMT>(c[u], step[u]);
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

hipError_t launch_page_any(bool write, const PageLayout& l, const PageParams& p, hipStream_t stream) {
    if (l.d == 64)
        return l.format == 0   ? launch_page<0, 64>(write, p, stream)
               : l.format == 1 ? launch_page<1, 64>(write, p, stream)
                               : launch_page<2, 64>(write, p, stream);
    return l.format == 0   ? launch_page<0, 128>(write, p, stream)
           : l.format == 1 ? launch_page<1, 128>(write, p, stream)
                           : launch_page<2, 128>(write, p, stream);
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

// append_kernels.hip - norms and rotation of new queries and keys, and the
// write of the keys and values into a paged cache, in one pass, for gfx950.
//
// A workgroup takes whole tokens, as the rotation alone does: a thread per
// (token, pair) forms the angle in binary64 and leaves its cosine and sine in
// LDS, then d / 16 lanes take a vector, 8 pairs each. Queries go out as rows.
// A key is rounded to bf16 as it would be on its way through memory (so the
// pages hold the bytes that rotation and write give one after the other) and
// quantised by the lanes that hold it; a value goes from its row to its codes.
// The maximum that 8-bit codes need is over the whole vector, in whatever order
// the lanes hold it. A block of 32 channels of 4-bit codes is not: there the lanes of a
// key change their chunks for those of 16 channels in a row, through LDS.
//
// Bound: memory and, for two thirds of the time, vector instructions (300 for 8 vectors). 8191 tokens of 32 query and 16
// key and value heads of 128 out of the projection's rows, e4m3 pages: 40 us for 101 MB read and 84 MB written, 4.6 TB/s
// (rotation and write alone: 30 + 12 us). The weights, held packed in registers, and the slots, in LDS, were 5 us of
// loads that wait on one another. A step of 15 tokens: 5.3 us, a launch and three dependent reads (two launches: 6.8).
#include "attend.h"
#include "kernels_common.h"
#include "page_codes.h"

namespace kvc {
namespace {

constexpr int kDevBadSlot = 16;  // KVC_DEV_BAD_SLOT

struct AppendParams {
    RowsDev q_in, k_in, v_in, q_out;
    const uint16_t *q_weight, *k_weight;
    const int64_t* positions;
    const int64_t* slots;
    uint8_t* pages;
    int32_t* status;
    uint64_t steps, page_bytes;
    uint32_t n, Hq, Hk, page_shift, num_pages;
    uint32_t n_pairs, pairing;
    float eps;
    float f[kMaxPairs];
};

typedef __attribute__((address_space(1))) kvc_u32x4 global_u32x4;

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}
__device__ __forceinline__ kvc_u32x4 vec4(const uint4& x) { return kvc_u32x4{x.x, x.y, x.z, x.w}; }

// sum over the LPV (4 or 8) lanes of a vector
template <int LPV>
__device__ __forceinline__ float sum_lanes(float v) {
    v += dpp_xor1(v);
    v += dpp_xor2(v);
    if (LPV == 8)  // row_half_mirror: the other four lanes of eight
        v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xF, 0xF, true));
    return v;
}

template <int FMT, int D, int TW>
__global__ __launch_bounds__(kBlockThreads) void append_kernel(AppendParams p) {
    fetch_arguments<sizeof(AppendParams)>();
    constexpr uint32_t LPV = D / 16;
    constexpr uint32_t VPB = kBlockThreads / LPV;  // vectors at a time
    __shared__ float cs[TW][kMaxPairs], sn[TW][kMaxPairs];
    __shared__ int64_t slots[TW];
    __shared__ uint4 turn_about[FMT == kPageFp4 ? kBlockThreads * 2 : 1];
    const uint32_t tok0 = blockIdx.x * TW;
    const uint32_t ntok = p.n - tok0 < TW ? p.n - tok0 : TW;
    const uint32_t heads = p.Hq + 2 * p.Hk;
    const uint32_t i = threadIdx.x % LPV;
    const uint32_t nrot = p.n_pairs / 8;  // lanes of a vector that hold pairs
    const bool turned = i < nrot;
    // the lane's two chunks of 8 channels: of a value always 16 in a row
    const uint32_t oa = turned && p.pairing == 0 ? 8 * i : 16 * i;
    const uint32_t ob = turned && p.pairing == 0 ? p.n_pairs + 8 * i : 16 * i + 8;
    kvc_u32x4 wq[2] = {}, wk[2] = {};
    if (p.q_weight) {
        wq[0] = *reinterpret_cast<const kvc_u32x4*>(p.q_weight + oa);
        wq[1] = *reinterpret_cast<const kvc_u32x4*>(p.q_weight + ob);
    }
    if (p.k_weight) {
        wk[0] = *reinterpret_cast<const kvc_u32x4*>(p.k_weight + oa);
        wk[1] = *reinterpret_cast<const kvc_u32x4*>(p.k_weight + ob);
    }
    uint32_t t = 0, h = threadIdx.x / LPV;
    const auto settle = [&]() {
        while (h >= heads && t < ntok) {
            h -= heads;
            ++t;
        }
    };
    kvc_u32x4 xa{}, xb{};
    const auto load = [&]() {
        if (t >= ntok) return;
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hk;
        const uint64_t data = is_q ? (uint64_t)p.q_in.data : is_v ? (uint64_t)p.v_in.data : (uint64_t)p.k_in.data;
        const uint64_t ts = is_q ? p.q_in.ts : is_v ? p.v_in.ts : p.k_in.ts;
        const uint64_t hs = is_q ? p.q_in.hs : is_v ? p.v_in.hs : p.k_in.hs;
        const uint32_t head = is_q ? h : is_v ? h - p.Hq - p.Hk : h - p.Hq;
        const uint64_t x = data + 2 * ((tok0 + t) * ts + head * hs);
        xa = *(const global_u32x4*)(x + 2 * (is_v ? 16 * i : oa));
        xb = *(const global_u32x4*)(x + 2 * (is_v ? 16 * i + 8 : ob));
    };
    settle();
    load();
    if (threadIdx.x < ntok) slots[threadIdx.x] = p.slots[tok0 + threadIdx.x];
    for (uint32_t j = threadIdx.x; j < TW * kMaxPairs; j += kBlockThreads) {
        const uint32_t jt = j / kMaxPairs, pair = j % kMaxPairs;
        if (jt < ntok && pair < p.n_pairs) {
            const double turns = (double)p.positions[tok0 + jt] * (double)p.f[pair] * 0.15915494309189533577;
            const float r = 2.0f * (float)(turns - rint(turns));
            float s, c;
            sincospif(r, &s, &c);
            cs[jt][pair] = c;
            sn[jt][pair] = s;
        }
    }
    __syncthreads();
    while (t < ntok) {
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hk;
        const uint32_t head = is_q ? h : is_v ? h - p.Hq - p.Hk : h - p.Hq;
        const uint32_t t_now = t;
        uint4 ya = make_uint4(xa.x, xa.y, xa.z, xa.w), yb = make_uint4(xb.x, xb.y, xb.z, xb.w);
        const int64_t slot = slots[t];
        h += VPB;
        settle();
        load();
        if (!is_v) {
            float a[8], b[8];
            unpack8(ya, a);
            unpack8(yb, b);
            if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
                float ss = 0.0f;
#pragma unroll
                for (int u = 0; u < 8; ++u) ss = fmaf(a[u], a[u], fmaf(b[u], b[u], ss));
                ss = sum_lanes<LPV>(ss);
                const float inv = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
                float w[8];
                { const kvc_u32x4 z = is_q ? wq[0] : wk[0]; unpack8(make_uint4(z.x, z.y, z.z, z.w), w); }
#pragma unroll
                for (int u = 0; u < 8; ++u) a[u] = a[u] * inv * w[u];
                { const kvc_u32x4 z = is_q ? wq[1] : wk[1]; unpack8(make_uint4(z.x, z.y, z.z, z.w), w); }
#pragma unroll
                for (int u = 0; u < 8; ++u) b[u] = b[u] * inv * w[u];
            }
            if (turned) {
                float c[8], s[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    c[u] = cs[t_now][8 * i + u];
                    s[u] = sn[t_now][8 * i + u];
                }
                if (p.pairing == 0) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const float ra = fmaf(a[u], c[u], -(b[u] * s[u])), rb = fmaf(a[u], s[u], b[u] * c[u]);
                        a[u] = ra;
                        b[u] = rb;
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float ra = fmaf(a[2 * u], c[u], -(a[2 * u + 1] * s[u]));
                        const float rb = fmaf(a[2 * u], s[u], a[2 * u + 1] * c[u]);
                        a[2 * u] = ra;
                        a[2 * u + 1] = rb;
                        const float rc = fmaf(b[2 * u], c[4 + u], -(b[2 * u + 1] * s[4 + u]));
                        const float rd = fmaf(b[2 * u], s[4 + u], b[2 * u + 1] * c[4 + u]);
                        b[2 * u] = rc;
                        b[2 * u + 1] = rd;
                    }
                }
            }
            ya = pack8(a);
            yb = pack8(b);
        }
        if (is_q) {
            uint16_t* y = p.q_out.data + (tok0 + t_now) * p.q_out.ts + head * p.q_out.hs;
            if (TW > 1) {
                __builtin_nontemporal_store(vec4(ya), (global_u32x4*)(uint64_t)(y + oa));
                __builtin_nontemporal_store(vec4(yb), (global_u32x4*)(uint64_t)(y + ob));
            } else {
                *(global_u32x4*)(uint64_t)(y + oa) = vec4(ya);
                *(global_u32x4*)(uint64_t)(y + ob) = vec4(yb);
            }
            continue;
        }
        // ---- into the page of the token's slot
        const bool inside = slot >= 0 && (uint64_t)slot < (uint64_t)p.num_pages << p.page_shift;
        if (slot >= 0 && !inside && p.status) atomicOr(p.status, kDevBadSlot);
        const uint64_t s = inside ? (uint64_t)slot : 0;
        const uint64_t line = ((uint64_t)(is_v ? p.Hk + head : head) << p.page_shift) + (s & ((1u << p.page_shift) - 1));
        uint8_t* page = p.pages + (s >> p.page_shift) * p.page_bytes;
        uint8_t* codes = page + line * page_code_bytes(FMT, D);
        uint8_t* step_at = page + p.steps + line * page_step_bytes(FMT, D);
        const uint32_t ca = is_v ? 16 * i : oa, cb = is_v ? 16 * i + 8 : ob;
        if constexpr (FMT == kPageBf16) {
            if (inside) {
                *reinterpret_cast<uint4*>(codes + 2 * ca) = ya;
                *reinterpret_cast<uint4*>(codes + 2 * cb) = yb;
            }
        } else if constexpr (FMT == kPageFp4) {
            if (!is_v && p.pairing == 0 && nrot) {
                // chunks by channel, in the vector's own place: its lanes are of one wave, which runs LDS in order
                uint4* x = turn_about + (threadIdx.x / LPV) * (D / 8);
                x[ca / 8] = ya;
                x[cb / 8] = yb;
                __builtin_amdgcn_wave_barrier();
                ya = x[2 * i];
                yb = x[2 * i + 1];
                __builtin_amdgcn_wave_barrier();
            }
            const uint32_t ma = magnitude8(ya), mb = magnitude8(yb);
            uint32_t power;
            const uint32_t m = max_lanes<2>(ma > mb ? ma : mb);
            const uint2 c = make_uint2(quantise8_fp4(ya, m, power), quantise8_fp4(yb, m, power));
            if (inside) {
                *reinterpret_cast<uint2*>(codes + 8 * i) = c;
                if (i % 2 == 0) step_at[i / 2] = (uint8_t)power;
            }
        } else {
            const uint32_t ma = magnitude8(ya), mb = magnitude8(yb);
            const uint32_t m = max_lanes<LPV>(ma > mb ? ma : mb);
            float step;
            const uint2 c = quantise8<FMT>(ya, m, step), d = quantise8<FMT>(yb, m, step);
            if (inside) {
                *reinterpret_cast<uint2*>(codes + ca) = c;
                *reinterpret_cast<uint2*>(codes + cb) = d;
                if (i == 0) *reinterpret_cast<float*>(step_at) = step;
            }
        }
    }
}

// Four tokens a workgroup (every thread an angle) and stores past the caches from 4096 tokens on, below one token: 8191
// tokens with one, two, four, eight 54.4, 51.3, 52.3 and 51.8 us (bf16 pages, with the read-back), heads of 64 40.5, 28.5,
// 28.0 and 27.3; 4096 31.3, 25.1, 24.7 and 28.2; 1000 tokens, 11.9 with any.
template <int FMT, int D>
hipError_t launch(const AppendParams& p, hipStream_t stream) {
    if (p.n >= 4096) return launch_kernel(append_kernel<FMT, D, 4>, dim3((p.n + 3) / 4), dim3(kBlockThreads), stream, p);
    return launch_kernel(append_kernel<FMT, D, 1>, dim3(p.n), dim3(kBlockThreads), stream, p);
}
template <int D>
hipError_t launch_of(uint32_t format, const AppendParams& p, hipStream_t stream) {
    switch (format) {
        case kPageBf16: return launch<kPageBf16, D>(p, stream);
        case kPageInt8: return launch<kPageInt8, D>(p, stream);
        case kPageFp8: return launch<kPageFp8, D>(p, stream);
        default: return launch<kPageFp4, D>(p, stream);
    }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, hipStream_t stream) {
    AppendParams p{};
    p.q_in = a.q_in;
    p.k_in = a.k_in;
    p.v_in = a.v_in;
    p.q_out = a.q_out;
    p.q_weight = static_cast<const uint16_t*>(a.q_weight);
    p.k_weight = static_cast<const uint16_t*>(a.k_weight);
    p.positions = a.positions;
    p.slots = a.slots;
    p.pages = a.pages;
    p.status = a.status;
    p.steps = a.lay.steps;
    p.page_bytes = a.lay.page_bytes;
    p.n = a.n;
    p.Hq = a.Hq;
    p.Hk = a.lay.H;
    p.page_shift = 31 - __builtin_clz(a.lay.P);
    p.num_pages = a.lay.num_pages;
    p.n_pairs = a.n_pairs;
    p.pairing = a.pairing;
    p.eps = a.eps;
    for (uint32_t j = 0; j < a.n_pairs; ++j) p.f[j] = a.inv_freq[j];
    return a.lay.d == 64 ? launch_of<64>(a.lay.format, p, stream) : launch_of<128>(a.lay.format, p, stream);
}

}  // namespace kvc
